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
// Bound by HBM: o and g in, y out, about 12 operations an entry (26 in the gradients).
// A group of d / 8 lanes holds one row in registers (the mean and the sum of squares
// are two passes over registers, not a difference of sums).  A CTA keeps one head and
// walks tokens, so w and the sums for dw stay in registers, and the addresses of a
// token's rows follow from the last one's.  Rows come four (bf16) ahead through the
// ring of rows.cuh: without it 6 to 12 rows' loads an SM were in flight and the
// gradients took 92 us, with it 66.  One GB300, bf16: 8 x 8192 tokens of 16 heads of
// 256 in 238 us (6.8 TB/s, the rate of a copy); gradients of 4 x 4093 tokens of 16
// heads of 128, centred, 59.5 us (5.6 TB/s; the kernel 57 of them, the sums over CTAs
// the rest), where the instructions (0.68 of the issue slots) bound it as well.
#include <algorithm>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kThreads = 128;
constexpr int kRingBytes = 8;  // rows of the ring: kRingBytes / sizeof(T)

// One tensor's addresses, in elements: head h's rows start at h_stride h, a walk's
// next token lies `step` further, and `wrap` more where that is past the sequence's end.
struct Rows {
    const void* p;
    long long b, t, h;  // strides
    long long step, wrap;
};

struct GateParams {
    Rows o, gate, dy, y, d_o, d_gate;  // gate.p may be null
    const float* w;
    float* part;         // [tokens' blocks][H][d] or null
    Divide by_T;
    unsigned tokens;     // B T
    unsigned leap_t;     // tokens from one to the walk's next, modulo T
    int H, d, center;
    float eps;
};

// A place in one tensor that walks with the tokens.
template <typename T>
struct Cursor {
    T* at;

    __device__ __forceinline__ Cursor(const Rows& r, int h, unsigned b, unsigned t)
        : at((T*)r.p + h * r.h + b * r.b + t * r.t) {}
    __device__ __forceinline__ void next(const Rows& r, bool wrapped) {
        at += r.step;
        if (wrapped) at += r.wrap;
    }
};

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
__global__ void __launch_bounds__(kThreads, BWD ? 5 : 6) head_gate_kernel(const __grid_constant__ GateParams p) {
    constexpr int kGroups = kThreads / G, kRing = kRingBytes / (int)sizeof(T), kSlot = 8 * G;
    __shared__ __align__(16) T ring[kRing][BWD ? 3 : 2][kGroups * kSlot];  // o, gate, dy
    if (BWD) tc::griddep_launch_dependents();  // the sums' kernel may be scheduled (it waits itself)
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, e = lane * 8, h = blockIdx.x;
    const bool on = e < p.d;
    const float inv_d = 1.f / (float)p.d;
    const bool gated = p.gate.p != nullptr;
    const unsigned leap = gridDim.y * kGroups, first = blockIdx.y * kGroups + grp;
    unsigned b0, t0;
    p.by_T(first, &b0, &t0);

    Cursor<const T> o(p.o, h, b0, t0), gate(p.gate, h, b0, t0), dy(p.dy, h, b0, t0);
    unsigned f_m = first, f_t = t0;
    int f_slot = 0;
    auto fetch = [&]() {
        if (f_m - grp < p.tokens) {  // the same for every group
            const bool there = f_m < p.tokens;
            copy_row<T, G>(&ring[f_slot][0][grp * kSlot], there ? o.at : (const T*)p.o.p, lane, p.d, there);
            if (gated)
                copy_row<T, G>(&ring[f_slot][1][grp * kSlot], there ? gate.at : (const T*)p.gate.p, lane, p.d,
                               there);
            if (BWD)
                copy_row<T, G>(&ring[f_slot][BWD ? 2 : 0][grp * kSlot], there ? dy.at : (const T*)p.dy.p, lane,
                               p.d, there);
            f_m += leap;
            f_t += p.leap_t;
            const bool wrapped = f_t >= p.by_T.T;
            if (wrapped) f_t -= p.by_T.T;
            o.next(p.o, wrapped);
            gate.next(p.gate, wrapped);
            if (BWD) dy.next(p.dy, wrapped);
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
    Cursor<T> y(BWD ? p.d_o : p.y, h, b0, t0), d_gate(p.d_gate, h, b0, t0);
    unsigned t = t0;
    int slot = 0;
    for (unsigned m = first; m - grp < p.tokens; m += leap) {
        const bool row_on = on && m < p.tokens;
        copies_wait<kRing - 1>();
        __syncwarp();
        float2 n[4], g[4], du[4];
        floats8<false>(raw8<true>(&ring[slot][0][grp * kSlot], e, e + 4), n);
        if (gated) floats8<false>(raw8<true>(&ring[slot][1][grp * kSlot], e, e + 4), g);
        if (BWD) floats8<false>(raw8<true>(&ring[slot][BWD ? 2 : 0][grp * kSlot], e, e + 4), du);
        __syncwarp();
        fetch();
        slot = slot + 1 == kRing ? 0 : slot + 1;
        const float r = norm_row<G>(n, on, p.center, inv_d, p.eps);
        if (!BWD) {
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] = __fmul2_rn(n[j], w[j]);
            if (gated) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    n[j] = __fmul2_rn(n[j], __fmul2_rn(g[j], make_float2(sigmoid<T>(g[j].x), sigmoid<T>(g[j].y))));
            }
            if (row_on) store8<true, false>(y.at, e, e + 4, n);
        } else {
            if (gated) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 sg = make_float2(sigmoid<T>(g[j].x), sigmoid<T>(g[j].y));
                    // the gate's slope: sigma + g sigma (1 - sigma)
                    const float2 act = __fmul2_rn(g[j], sg);
                    const float2 slope = __ffma2_rn(act, __ffma2_rn(sg, both(-1.f), both(1.f)), sg);
                    g[j] = __fmul2_rn(__fmul2_rn(du[j], __fmul2_rn(n[j], w[j])), slope);
                    du[j] = __fmul2_rn(du[j], act);
                }
                if (row_on) store8<true, false>(d_gate.at, e, e + 4, g);
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
            if (row_on) store8<true, false>(y.at, e, e + 4, du);
        }
        t += p.leap_t;
        const bool wrapped = t >= p.by_T.T;
        if (wrapped) t -= p.by_T.T;
        y.next(BWD ? p.d_o : p.y, wrapped);
        if (BWD) d_gate.next(p.d_gate, wrapped);
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
constexpr int kFwdPerSm = 48, kBwdPerSm = 10;

unsigned token_blocks(const HeadGateArgs& a, bool bwd) {
    const long long groups = kThreads / group_lanes(a.d);
    const long long turns = ((long long)a.B * a.T + groups - 1) / groups;
    const long long most = ((long long)sm_count() * (bwd ? kBwdPerSm : kFwdPerSm) + a.H - 1) / a.H;
    return (unsigned)std::min(turns, std::min(most, 65535ll));
}

GateParams params(const HeadGateArgs& a, unsigned blocks) {
    const unsigned leap = blocks * (unsigned)(kThreads / group_lanes(a.d));
    const long long leap_b = leap / (unsigned)a.T, leap_t = leap % (unsigned)a.T;
    auto rows = [&](const void* p, long long b, long long t, long long h) {
        return Rows{p, b, t, h, leap_b * b + leap_t * t, b - a.T * t};
    };
    auto heads_first = [&](const void* p, const long long* s) { return rows(p, s[0], s[2], s[1]); };
    auto tokens_first = [&](const void* p, const long long* s) { return rows(p, s[0], s[1], s[2]); };
    GateParams p;
    p.o = heads_first(a.o, a.o_strides);
    p.gate = tokens_first(a.gate, a.gate_strides);
    p.dy = tokens_first(a.dy, a.dy_strides);
    p.y = tokens_first(a.y, a.y_strides);
    p.d_o = heads_first(a.d_o, a.do_strides);
    p.d_gate = tokens_first(a.d_gate, a.dgate_strides);
    p.w = a.weight;
    p.part = a.d_weight ? (float*)a.workspace : nullptr;
    p.by_T = Divide::by(a.T);
    p.tokens = (unsigned)((long long)a.B * a.T);
    p.leap_t = (unsigned)leap_t;
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
    const dim3 grid(a.H, token_blocks(a, false));
    const GateParams p = params(a, grid.y);
    TraceScope trace("head_gate_fwd_kernel", s);
    if (a.bf16) launch<__nv_bfloat16>(p, false, grid, s);
    else launch<float>(p, false, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_head_gate_bwd(const HeadGateArgs& a, cudaStream_t s) {
    const dim3 grid(a.H, token_blocks(a, true));
    const GateParams p = params(a, grid.y);
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
