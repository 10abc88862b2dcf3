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
#include "trace.h"

namespace la {

namespace {

constexpr int kThreads = 256;

struct GateParams {
    const void *o, *gate, *dy;
    void *y, *d_o, *d_gate;
    const float* w;
    float* part;  // [tokens' blocks][H][d] or null
    long long o_sb, o_sh, o_st, g_sb, g_st, g_sh, dy_sb, dy_st, dy_sh;
    long long y_sb, y_st, y_sh, do_sb, do_sh, do_st, dg_sb, dg_st, dg_sh;
    unsigned tokens;  // B T
    int T, H, d, center;
    float eps;
};

// sigma(g), with no overflow turned into a NaN: e^-g = inf gives 0.
__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + expf(-g)); }

// x <- its normed row, returns r.  Lanes past the row hold zeros and keep them.
template <int G>
__device__ __forceinline__ float norm_row(float (&x)[8], bool on, int center, float inv_d, float eps) {
    if (center) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += x[j];
        const float mean = group_sum<G>(sum) * inv_d;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = on ? x[j] - mean : 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
    const float r = rsqrtf(group_sum<G>(ss) * inv_d + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= r;
    return r;
}

// Grid: (heads, blocks of tokens).
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) head_gate_fwd_kernel(const __grid_constant__ GateParams p) {
    constexpr int kGroups = kThreads / G;
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, e = lane * 8, h = blockIdx.x;
    const bool on = e < p.d;
    const float inv_d = 1.f / (float)p.d;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = p.w && on ? __ldg(p.w + (size_t)h * p.d + e + j) : 1.f;
    for (unsigned base = blockIdx.y * kGroups; base < p.tokens; base += gridDim.y * kGroups) {
        const unsigned m = base + grp;
        const bool row_on = on && m < p.tokens;
        const int b = (int)(m / (unsigned)p.T), t = (int)(m - (unsigned)b * (unsigned)p.T);
        Raw8<T> ro = zero_raw8<T>(), rg = zero_raw8<T>();
        if (row_on) {
            ro = load_raw8<true>((const T*)p.o + b * p.o_sb + h * p.o_sh + t * p.o_st, e, e + 4);
            if (p.gate)
                rg = load_raw8<true>((const T*)p.gate + b * p.g_sb + t * p.g_st + h * p.g_sh, e, e + 4);
        }
        float x[8], g[8];
        floats8(ro, x);
        floats8(rg, g);
        norm_row<G>(x, on, p.center, inv_d, p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] *= w[j];
            if (p.gate) x[j] *= g[j] * sigmoid(g[j]);
        }
        if (row_on)
            store8<true>((T*)p.y + b * p.y_sb + t * p.y_st + h * p.y_sh, e, e + 4, x);
    }
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) head_gate_bwd_kernel(const __grid_constant__ GateParams p) {
    constexpr int kGroups = kThreads / G;
    __shared__ float red[kThreads * 8];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, e = lane * 8, h = blockIdx.x;
    const bool on = e < p.d;
    const float inv_d = 1.f / (float)p.d;
    float w[8], dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        w[j] = p.w && on ? __ldg(p.w + (size_t)h * p.d + e + j) : 1.f;
        dw[j] = 0.f;
    }
    for (unsigned base = blockIdx.y * kGroups; base < p.tokens; base += gridDim.y * kGroups) {
        const unsigned m = base + grp;
        const bool row_on = on && m < p.tokens;
        const int b = (int)(m / (unsigned)p.T), t = (int)(m - (unsigned)b * (unsigned)p.T);
        Raw8<T> ro = zero_raw8<T>(), rg = zero_raw8<T>(), rd = zero_raw8<T>();
        if (row_on) {
            ro = load_raw8<true>((const T*)p.o + b * p.o_sb + h * p.o_sh + t * p.o_st, e, e + 4);
            rd = load_raw8<true>((const T*)p.dy + b * p.dy_sb + t * p.dy_st + h * p.dy_sh, e, e + 4);
            if (p.gate)
                rg = load_raw8<true>((const T*)p.gate + b * p.g_sb + t * p.g_st + h * p.g_sh, e, e + 4);
        }
        float n[8], g[8], du[8];
        floats8(ro, n);
        floats8(rd, du);
        floats8(rg, g);
        const float r = norm_row<G>(n, on, p.center, inv_d, p.eps);
        float dot = 0.f, mean = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (p.gate) {
                const float sg = sigmoid(g[j]), d = du[j];
                du[j] = d * (g[j] * sg);
                g[j] = d * n[j] * w[j] * (sg * (1.f + g[j] * (1.f - sg)));
            }
            if (row_on) dw[j] += du[j] * n[j];
            du[j] *= w[j];
            dot += du[j] * n[j];
            mean += du[j];
        }
        dot = group_sum<G>(dot) * inv_d;
        mean = p.center ? group_sum<G>(mean) * inv_d : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) du[j] = r * (du[j] - mean - n[j] * dot);
        if (row_on) {
            store8<true>((T*)p.d_o + b * p.do_sb + h * p.do_sh + t * p.do_st, e, e + 4, du);
            if (p.gate)
                store8<true>((T*)p.d_gate + b * p.dg_sb + t * p.dg_st + h * p.dg_sh, e, e + 4, g);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (on) red[grp * G * 8 + e + j] = dw[j];
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += kThreads) {
        float sum = 0.f;
        for (int i = 0; i < kGroups; ++i) sum += red[i * G * 8 + c];
        p.part[((size_t)blockIdx.y * p.H + h) * p.d + c] = sum;
    }
}

// Blocks of tokens a head's CTAs share: enough CTAs to fill the card a few times.
unsigned token_blocks(const HeadGateArgs& a, int per_sm) {
    const long long groups = kThreads / group_lanes(a.d), tokens = (long long)a.B * a.T;
    const long long want = ((long long)sm_count() * per_sm + a.H - 1) / a.H;
    return (unsigned)std::min<long long>(std::min<long long>((tokens + groups - 1) / groups, want), 65535);
}

constexpr int kFwdPerSm = 32, kBwdPerSm = 8;

GateParams params(const HeadGateArgs& a) {
    GateParams p;
    p.o = a.o; p.gate = a.gate; p.dy = a.dy;
    p.y = a.y; p.d_o = a.d_o; p.d_gate = a.d_gate;
    p.w = a.weight;
    p.part = a.d_weight ? (float*)a.workspace : nullptr;
    p.o_sb = a.o_strides[0]; p.o_sh = a.o_strides[1]; p.o_st = a.o_strides[2];
    p.g_sb = a.gate_strides[0]; p.g_st = a.gate_strides[1]; p.g_sh = a.gate_strides[2];
    p.dy_sb = a.dy_strides[0]; p.dy_st = a.dy_strides[1]; p.dy_sh = a.dy_strides[2];
    p.y_sb = a.y_strides[0]; p.y_st = a.y_strides[1]; p.y_sh = a.y_strides[2];
    p.do_sb = a.do_strides[0]; p.do_sh = a.do_strides[1]; p.do_st = a.do_strides[2];
    p.dg_sb = a.dgate_strides[0]; p.dg_st = a.dgate_strides[1]; p.dg_sh = a.dgate_strides[2];
    p.tokens = (unsigned)((long long)a.B * a.T);
    p.T = a.T; p.H = a.H; p.d = a.d; p.center = a.center;
    p.eps = a.eps;
    return p;
}

template <typename T, int G>
void launch(const GateParams& p, bool bwd, dim3 grid, cudaStream_t s) {
    if (bwd) head_gate_bwd_kernel<T, G><<<grid, kThreads, 0, s>>>(p);
    else head_gate_fwd_kernel<T, G><<<grid, kThreads, 0, s>>>(p);
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
    return (size_t)token_blocks(a, kBwdPerSm) * a.H * a.d * sizeof(float);
}

cudaError_t launch_head_gate_fwd(const HeadGateArgs& a, cudaStream_t s) {
    const GateParams p = params(a);
    const dim3 grid(a.H, token_blocks(a, kFwdPerSm));
    TraceScope trace("head_gate_fwd_kernel", s);
    if (a.bf16) launch<__nv_bfloat16>(p, false, grid, s);
    else launch<float>(p, false, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_head_gate_bwd(const HeadGateArgs& a, cudaStream_t s) {
    const GateParams p = params(a);
    const dim3 grid(a.H, token_blocks(a, kBwdPerSm));
    {
        TraceScope trace("head_gate_bwd_kernel", s);
        if (a.bf16) launch<__nv_bfloat16>(p, true, grid, s);
        else launch<float>(p, true, grid, s);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    return launch_partial_sum(p.part, (int)grid.y, a.d_weight, a.H * a.d, nullptr, 0, s);
}

}  // namespace la
