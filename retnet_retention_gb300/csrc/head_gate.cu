// The norm and gate of each head's output, [B][H][T][d] (any strides: retention's
// layout, or the recurrence's [B][T][H][d]) to the layer's row [B][T][H][d]:
//
//   n = (o - mean o) r, r = (mean (o - mean o)^2 + eps)^(-1/2)   (no mean taken out
//                                                                 unless centred)
//   y = n w g sigmoid(g)                                         (w, g optional)
//
// and its gradients: du = dy g sigma, dg = dy n w sigma (1 + g (1 - sigma)),
// dw = sum du n over the tokens, dn = du w,
// do = r (dn - [mean dn] - n mean(dn n)).
//
// Bound by HBM: o and g in, y out, about 12 operations an entry.  A group of d / 8
// lanes holds one row in registers (the mean and the sum of squares are two passes
// over registers, not a difference of sums).  A CTA keeps one head and walks
// tokens, so w and the sums for dw stay in registers.
#include <algorithm>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kThreads = 128;
constexpr int kRingBytes = 8;  // rows of the ring: kRingBytes / sizeof(T)

struct GateParams {
    const void *o, *gate, *dy;
    void *y, *d_o, *d_gate;
    const float* w;
    float* part;  // [tokens' blocks][H][d] or null
    long long o_b, o_h, o_t, g_b, g_t, g_h, dy_b, dy_t, dy_h;
    long long y_b, y_t, y_h, do_b, do_h, do_t, dg_b, dg_t, dg_h;
    Divide by_T;
    unsigned tokens;  // B T
    int H, d, center;
    float eps;
};

// sigma(g) to a few ulp: e^-g may overflow to infinity, whose reciprocal is 0.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + expf(-g)); }

// x <- its normed row, returns r.  Lanes past the row hold zeros and keep them.
template <int G>
__device__ __forceinline__ float norm_row(float2 (&x)[4], bool on, int center, float inv_d, float eps) {
    if (center) {
        const float2 sum = __fadd2_rn(__fadd2_rn(x[0], x[1]), __fadd2_rn(x[2], x[3]));
        float mean = group_sum<G>(sum.x + sum.y) * inv_d;
        if (!on) mean = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fadd2_rn(x[j], both(-mean));
    }
    const float r = rsqrtf(group_sum<G>(dot8(x, x)) * inv_d + eps);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(x[j], both(r));
    return r;
}

// Grid: (heads, blocks of tokens).
template <typename T, int G, bool BWD>
__global__ void __launch_bounds__(kThreads, 6) head_gate_kernel(const __grid_constant__ GateParams p) {
    constexpr int kGroups = kThreads / G, kRing = kRingBytes / (int)sizeof(T), kSlot = 8 * G;
    __shared__ __align__(16) T ring[kRing][BWD ? 3 : 2][kGroups * kSlot];  // o, gate, dy
    if (BWD) tc::griddep_launch_dependents();  // the sums' kernel may be scheduled (it waits itself)
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, e = lane * 8, h = blockIdx.x;
    const bool on = e < p.d;
    const float inv_d = 1.f / (float)p.d;
    const T* o = (const T*)p.o + h * p.o_h;
    const T* gate = p.gate ? (const T*)p.gate + h * p.g_h : nullptr;
    const T* dy = BWD ? (const T*)p.dy + h * p.dy_h : nullptr;
    const unsigned leap = gridDim.y * kGroups;

    unsigned f_base = blockIdx.y * kGroups;
    int f_slot = 0;
    auto fetch = [&]() {
        if (f_base < p.tokens) {
            const bool there = f_base + grp < p.tokens;
            unsigned b, t;
            p.by_T(there ? f_base + grp : 0, &b, &t);
            copy_row<T, G>(&ring[f_slot][0][grp * kSlot], o + b * p.o_b + t * p.o_t, lane, p.d, there);
            if (gate)
                copy_row<T, G>(&ring[f_slot][1][grp * kSlot], gate + b * p.g_b + t * p.g_t, lane, p.d, there);
            if (BWD)
                copy_row<T, G>(&ring[f_slot][BWD ? 2 : 0][grp * kSlot], dy + b * p.dy_b + t * p.dy_t, lane, p.d,
                               there);
            f_base += leap;
        }
        copies_commit();
        f_slot = f_slot + 1 == kRing ? 0 : f_slot + 1;
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch();

    float2 w[4], dw[4];
    row_weights<false>(p.w ? p.w + (size_t)h * p.d : nullptr, on, e, e + 4, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[j] = make_float2(0.f, 0.f);
    int slot = 0;
    for (unsigned base = blockIdx.y * kGroups; base < p.tokens; base += leap) {
        const bool row_on = on && base + grp < p.tokens;
        copies_wait<kRing - 1>();
        __syncwarp();
        float2 n[4], g[4], du[4];
        floats8<false>(raw8<true>(&ring[slot][0][grp * kSlot], e, e + 4), n);
        if (gate) floats8<false>(raw8<true>(&ring[slot][1][grp * kSlot], e, e + 4), g);
        if (BWD) floats8<false>(raw8<true>(&ring[slot][BWD ? 2 : 0][grp * kSlot], e, e + 4), du);
        __syncwarp();
        fetch();
        slot = slot + 1 == kRing ? 0 : slot + 1;
        unsigned b, t;
        p.by_T(base + grp, &b, &t);
        const float r = norm_row<G>(n, on, p.center, inv_d, p.eps);
        if (!BWD) {
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] = __fmul2_rn(n[j], w[j]);
            if (gate) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    n[j] = __fmul2_rn(n[j], __fmul2_rn(g[j], make_float2(sigmoid(g[j].x), sigmoid(g[j].y))));
            }
            if (row_on)
                store8<true, false>((T*)p.y + h * p.y_h + b * p.y_b + t * p.y_t, e, e + 4, n);
        } else {
            if (gate) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 sg = make_float2(sigmoid(g[j].x), sigmoid(g[j].y));
                    // slope: sigma (1 + g (1 - sigma))
                    const float2 slope = __fmul2_rn(
                        sg, __ffma2_rn(g[j], __fadd2_rn(both(1.f), make_float2(-sg.x, -sg.y)), both(1.f)));
                    const float2 act = __fmul2_rn(g[j], sg);
                    g[j] = __fmul2_rn(__fmul2_rn(du[j], __fmul2_rn(n[j], w[j])), slope);
                    du[j] = __fmul2_rn(du[j], act);
                }
                if (row_on)
                    store8<true, false>((T*)p.d_gate + h * p.dg_h + b * p.dg_b + t * p.dg_t, e, e + 4, g);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // rows that are not there hold zeros and add none
                dw[j] = __ffma2_rn(du[j], n[j], dw[j]);
                du[j] = __fmul2_rn(du[j], w[j]);
            }
            const float along = -group_sum<G>(dot8(du, n)) * inv_d;
            float mean = 0.f;
            if (p.center) {
                const float2 sum = __fadd2_rn(__fadd2_rn(du[0], du[1]), __fadd2_rn(du[2], du[3]));
                mean = -group_sum<G>(sum.x + sum.y) * inv_d;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                du[j] = __fmul2_rn(both(r), __ffma2_rn(n[j], both(along), __fadd2_rn(du[j], both(mean))));
            if (row_on) store8<true, false>((T*)p.d_o + h * p.do_h + b * p.do_b + t * p.do_t, e, e + 4, du);
        }
    }
    if (!BWD || !p.part) return;
    float* red = reinterpret_cast<float*>(&ring[0][0][0]);
    static_assert(sizeof(ring) >= kThreads * 8 * sizeof(float), "a thread's eight sums fit the ring");
    copies_wait<0>();
    __syncthreads();
    if (on) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(&red[grp * kSlot + e + 2 * j]) = dw[j];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += kThreads) {
        float sum = 0.f;
        for (int i = 0; i < kGroups; ++i) sum += red[i * kSlot + c];
        p.part[((size_t)blockIdx.y * p.H + h) * p.d + c] = sum;
    }
}

// CTAs a head's tokens are shared out to: a few CTAs per SM in all; backward each
// leaves one row of partial sums.
constexpr int kFwdPerSm = 32, kBwdPerSm = 12;

unsigned token_blocks(const HeadGateArgs& a, bool bwd) {
    const long long groups = kThreads / group_lanes(a.d);
    const long long turns = ((long long)a.B * a.T + groups - 1) / groups;
    const long long most = ((long long)sm_count() * (bwd ? kBwdPerSm : kFwdPerSm) + a.H - 1) / a.H;
    return (unsigned)std::min(turns, std::min(most, 65535ll));
}

GateParams params(const HeadGateArgs& a) {
    GateParams p;
    p.o = a.o; p.gate = a.gate; p.dy = a.dy;
    p.y = a.y; p.d_o = a.d_o; p.d_gate = a.d_gate;
    p.w = a.weight;
    p.part = a.d_weight ? (float*)a.workspace : nullptr;
    p.o_b = a.o_strides[0]; p.o_h = a.o_strides[1]; p.o_t = a.o_strides[2];
    p.g_b = a.gate_strides[0]; p.g_t = a.gate_strides[1]; p.g_h = a.gate_strides[2];
    p.dy_b = a.dy_strides[0]; p.dy_t = a.dy_strides[1]; p.dy_h = a.dy_strides[2];
    p.y_b = a.y_strides[0]; p.y_t = a.y_strides[1]; p.y_h = a.y_strides[2];
    p.do_b = a.do_strides[0]; p.do_h = a.do_strides[1]; p.do_t = a.do_strides[2];
    p.dg_b = a.dgate_strides[0]; p.dg_t = a.dgate_strides[1]; p.dg_h = a.dgate_strides[2];
    p.tokens = (unsigned)((long long)a.B * a.T);
    p.by_T = Divide::by(a.T);
    p.H = a.H; p.d = a.d; p.center = a.center;
    p.eps = a.eps;
    return p;
}

template <typename T, int G>
void launch(const GateParams& p, bool bwd, dim3 grid, cudaStream_t s) {
    if (bwd) head_gate_kernel<T, G, true><<<grid, kThreads, 0, s>>>(p);
    else head_gate_kernel<T, G, false><<<grid, kThreads, 0, s>>>(p);
}

template <typename T>
void launch(const GateParams& p, bool bwd, dim3 grid, cudaStream_t s) {
    switch (group_lanes(p.d)) {
        case 2: launch<T, 2>(p, bwd, grid, s); break;
        case 4: launch<T, 4>(p, bwd, grid, s); break;
        case 8: launch<T, 8>(p, bwd, grid, s); break;
        case 16: launch<T, 16>(p, bwd, grid, s); break;
        default: launch<T, 32>(p, bwd, grid, s); break;
    }
}

}  // namespace

size_t head_gate_bwd_workspace_bytes(const HeadGateArgs& a) {
    return (size_t)token_blocks(a, true) * a.H * a.d * sizeof(float);
}

cudaError_t launch_head_gate_fwd(const HeadGateArgs& a, cudaStream_t s) {
    const GateParams p = params(a);
    const dim3 grid(a.H, token_blocks(a, false));
    TraceScope trace("head_gate_fwd_kernel", s);
    if (a.bf16) launch<__nv_bfloat16>(p, false, grid, s);
    else launch<float>(p, false, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_head_gate_bwd(const HeadGateArgs& a, cudaStream_t s) {
    const GateParams p = params(a);
    const dim3 grid(a.H, token_blocks(a, true));
    {
        TraceScope trace("head_gate_bwd_kernel", s);
        if (a.bf16) launch<__nv_bfloat16>(p, true, grid, s);
        else launch<float>(p, true, grid, s);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    return launch_partial_sum(p.part, (int)grid.y, a.d_weight, nullptr, 0, nullptr, a.H * a.d, s);
}

}  // namespace la
