// The per-channel gated recurrence over [B][T][D],
//
//   h_t = a_t h_(t-1) + x_t,   a_t = e^(log_a[b][t][c]),
//
// its gradients (c_t = a_t (dh_t + c_(t+1)), c_T = dh_T: dx_t = dh_t + c_(t+1),
// dlog_a_t = c_t h_(t-1), dh0 = c_0) and its single step.
//
// A run of tokens acts on the state as h -> A h + b, and two runs compose:
// (A2, b2) after (A1, b1) is (A2 A1, A2 b1 + b2).  So a round of tokens is split
// over the warps of a CTA and the CTAs of a cluster: every thread composes the rows
// it holds in registers, the runs' (A, b) are composed across warps (shared memory)
// and across the cluster's CTAs (each pushes its own into the others' shared
// memory, one cluster barrier a round), and every thread then replays its rows from
// the state that enters them.  x and log_a are read once and h written once; no
// workspace, no atomics, no waits on memory, and the order of all sums is fixed by
// the launch shape.
//
// A decay of exactly zero (log_a = -inf) restarts its channel: the old state is
// dropped by a selection, not multiplied by zero, so that an infinity or a NaN in
// it does not pass.  (A run whose product underflows drops it the same way.)
//
// Bound by HBM: log_a 4, x 2, h 2 bytes an entry (bf16).  State, products and sums
// are fp32; h is rounded where it is stored, never the state that is carried on.
#include <algorithm>

#include "rows.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;

struct ScanParams {
    const void* x;       // x, or dh in the backward walk
    const float* log_a;
    const float* s0;     // the state entering the walk (h0, or dh_T), or null
    const void* h_in;    // backward: the forward's h
    const float* h0;     // backward: the forward's initial state, or null
    void* y;             // h, or dx
    float* dlog_a;       // backward
    float* s_out;        // the state after the walk (h_T, or dh0), or null
    int T, D, tiles;     // tiles: channel tiles of a sequence
};

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_id() {
    unsigned r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// Write v to the same shared address in CTA `rank` of the cluster.
__device__ __forceinline__ void push(const float2* at, unsigned rank, float2 v) {
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(at);
    asm volatile(
        "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\t"
        "st.shared::cluster.v2.f32 [r], {%2, %3};\n\t}" ::"r"(a),
        "r"(rank), "f"(v.x), "f"(v.y)
        : "memory");
}

// The state s after a run (A, b).
__device__ __forceinline__ float after(float A, float b, float s) {
    return A == 0.f ? b : fmaf(A, s, b);
}

template <int V>
struct Pack;
template <>
struct Pack<1> {
    using F = float;
    using H = uint16_t;
};
template <>
struct Pack<2> {
    using F = float2;
    using H = uint32_t;
};

template <int V>
__device__ __forceinline__ void load_row(const float* p, float (&v)[V]) {
    const typename Pack<V>::F r = __ldg(reinterpret_cast<const typename Pack<V>::F*>(p));
    const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = f[j];
}
template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&v)[V]) {
    const typename Pack<V>::H r = __ldg(reinterpret_cast<const typename Pack<V>::H*>(p));
    v[0] = __uint_as_float((uint32_t)r << 16);
    if (V == 2) v[V - 1] = __uint_as_float((uint32_t)r & 0xffff0000u);
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
    typename Pack<V>::F r;
    float* f = reinterpret_cast<float*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = v[j];
    *reinterpret_cast<typename Pack<V>::F*>(p) = r;
}
template <int V>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&v)[V]) {
    if (V == 2) *reinterpret_cast<uint32_t*>(p) = bf16x2_bits(v[0], v[V - 1]);
    else *p = __float2bfloat16_rn(v[0]);
}

// One cluster walks one tile of 32 V channels of one sequence, R rows a thread and
// round; backward, it walks from the last token to the first.
template <typename T, int V, int R, bool BWD>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(const __grid_constant__ ScanParams p) {
    constexpr int C = 32 * V, kRun = kWarps * R;
    __shared__ float2 warp_run[2][kWarps][C];
    __shared__ float2 cta_run[2][kMaxCluster][C];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const unsigned rank = cluster_rank(), n = cluster_size(), unit = cluster_id();
    const unsigned b = unit / (unsigned)p.tiles, tile = unit - b * (unsigned)p.tiles;
    const int c0 = (int)tile * C + lane * V;
    const bool on = c0 < p.D;
    const size_t seq = (size_t)b * p.T * p.D + c0;
    const T* x = (const T*)p.x + seq;
    const T* h_in = (const T*)p.h_in + seq;
    const float* log_a = p.log_a + seq;
    T* y = (T*)p.y + seq;

    float state[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        state[j] = on && p.s0 ? p.s0[(size_t)b * p.D + c0 + j] : 0.f;
    if (n > 1) cluster_barrier();  // every CTA of the cluster runs before any is written to

    const int rounds = (int)(((long long)p.T + (long long)kRun * n - 1) / ((long long)kRun * n));
    for (int round = 0; round < rounds; ++round) {
        const int par = round & 1;
        const long long u0 = ((long long)round * n + rank) * kRun + w * R;  // first row, in walking order
        float a[R][V], v[R][V], hp[BWD ? R : 1][V];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const long long u = u0 + i;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                a[i][j] = 0.f;
                v[i][j] = 0.f;
                if (BWD) hp[BWD ? i : 0][j] = 0.f;
            }
            if (on && u < p.T) {
                const size_t t = BWD ? (size_t)(p.T - 1 - u) : (size_t)u;
                load_row<V>(log_a + t * p.D, a[i]);
                load_row<V>(x + t * p.D, v[i]);
                if (BWD) {
                    if (t > 0) load_row<V>(h_in + (t - 1) * p.D, hp[BWD ? i : 0]);
                    else if (p.h0) load_row<V>(p.h0 + (size_t)b * p.D + c0, hp[BWD ? i : 0]);
                }
            }
        }
        float A[V], bb[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.f, bb[j] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                a[i][j] = expf(a[i][j]);  // rows past the end: log_a 0, x 0 keep the state
                if (BWD) bb[j] = a[i][j] == 0.f ? 0.f : a[i][j] * (v[i][j] + bb[j]);
                else bb[j] = after(a[i][j], v[i][j], bb[j]);
                A[j] *= a[i][j];
            }
#pragma unroll
        for (int j = 0; j < V; ++j) warp_run[par][w][lane * V + j] = make_float2(A[j], bb[j]);
        __syncthreads();
        // the run before this warp's in the CTA, and the whole CTA's
        float pA[V], pb[V], tA[V], tb[V];
#pragma unroll
        for (int j = 0; j < V; ++j) tA[j] = 1.f, tb[j] = 0.f, pA[j] = 1.f, pb[j] = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 r = warp_run[par][i][lane * V + j];
                if (i == w) pA[j] = tA[j], pb[j] = tb[j];
                tb[j] = after(r.x, r.y, tb[j]);
                tA[j] *= r.x;
            }
        float s[V];
        if (n > 1) {
            for (unsigned to = w; to < n; to += kWarps)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    push(&cta_run[par][rank][lane * V + j], to, make_float2(tA[j], tb[j]));
            cluster_barrier();
            for (unsigned r = 0; r < n; ++r) {
                if (r == rank) {
#pragma unroll
                    for (int j = 0; j < V; ++j) s[j] = after(pA[j], pb[j], state[j]);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 g = cta_run[par][r][lane * V + j];
                    state[j] = after(g.x, g.y, state[j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[j] = after(pA[j], pb[j], state[j]);
                state[j] = after(tA[j], tb[j], state[j]);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const long long u = u0 + i;
            float out[V], dla[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (BWD) {
                    out[j] = v[i][j] + s[j];
                    s[j] = a[i][j] == 0.f ? 0.f : a[i][j] * out[j];
                    dla[j] = a[i][j] == 0.f ? 0.f : s[j] * hp[BWD ? i : 0][j];
                } else {
                    s[j] = after(a[i][j], v[i][j], s[j]);
                    out[j] = s[j];
                }
            }
            if (on && u < p.T) {
                const size_t t = BWD ? (size_t)(p.T - 1 - u) : (size_t)u;
                store_row<V>(y + t * p.D, out);
                if (BWD) store_row<V>(p.dlog_a + seq + t * p.D, dla);
            }
        }
    }
    if (p.s_out && on && rank == 0 && w == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.s_out[(size_t)b * p.D + c0 + j] = state[j];
    }
}

// h_out = a h_in + x, h = its rounding; four entries a thread.
template <typename T>
__global__ void __launch_bounds__(256) scan_step_kernel(const T* __restrict__ x,
                                                        const float* __restrict__ log_a,
                                                        const float* h_in, T* h, float* h_out,
                                                        size_t n4) {
    const size_t stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n4; i += stride) {
        const float4 l = __ldg(reinterpret_cast<const float4*>(log_a) + i);
        const float4 s = reinterpret_cast<const float4*>(h_in)[i];
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load_elem(x, i * 4 + j);
        const float4 o = make_float4(after(expf(l.x), v[0], s.x), after(expf(l.y), v[1], s.y),
                                     after(expf(l.z), v[2], s.z), after(expf(l.w), v[3], s.w));
        reinterpret_cast<float4*>(h_out)[i] = o;
        store_elem(h, i * 4, o.x);
        store_elem(h, i * 4 + 1, o.y);
        store_elem(h, i * 4 + 2, o.z);
        store_elem(h, i * 4 + 3, o.w);
    }
}

template <typename T, int V, int R, bool BWD>
cudaError_t launch(const ScanParams& p, int B, int cluster, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    const long long ctas = (long long)B * p.tiles * cluster;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scan_kernel<T, V, R, BWD>, p);
}

// Tiles of 64 channels where there are enough of them, of 32 otherwise, and CTAs of a
// cluster until the card is full or a CTA has a single round.
template <typename T, int R, bool BWD>
cudaError_t launch(ScanParams p, int B, cudaStream_t s) {
    const long long want = sm_count() * 2LL;
    const long long tiles2 = (p.D + 63) / 64, tiles1 = (p.D + 31) / 32;
    const bool wide = tiles2 * B * kMaxCluster >= want && p.D % 64 == 0;
    p.tiles = (int)(wide ? tiles2 : tiles1);
    int cluster = 1;
    while (cluster < kMaxCluster && (long long)p.tiles * B * cluster < want &&
           (long long)cluster * kWarps * R < p.T)
        cluster *= 2;
    return wide ? launch<T, 2, R, BWD>(p, B, cluster, s) : launch<T, 1, R, BWD>(p, B, cluster, s);
}

}  // namespace

cudaError_t launch_scan_fwd(const RecurrenceArgs& a, cudaStream_t s) {
    ScanParams p = {};
    p.x = a.x; p.log_a = a.log_a; p.s0 = a.h0; p.y = a.h; p.s_out = a.h_out;
    p.T = a.T; p.D = a.D;
    TraceScope trace("scan_kernel", s);
    const cudaError_t e = a.bf16 ? launch<__nv_bfloat16, 16, false>(p, a.B, s)
                                 : launch<float, 16, false>(p, a.B, s);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_scan_bwd(const RecurrenceArgs& a, cudaStream_t s) {
    ScanParams p = {};
    p.x = a.dh; p.log_a = a.log_a; p.s0 = a.dh_T; p.h_in = a.h; p.h0 = a.h0;
    p.y = a.dx; p.dlog_a = a.dlog_a; p.s_out = a.dh0;
    p.T = a.T; p.D = a.D;
    TraceScope trace("scan_bwd_kernel", s);
    const cudaError_t e = a.bf16 ? launch<__nv_bfloat16, 8, true>(p, a.B, s)
                                 : launch<float, 8, true>(p, a.B, s);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_scan_step(const RecurrenceArgs& a, cudaStream_t s) {
    const size_t n4 = (size_t)a.B * a.D / 4;
    const unsigned grid = (unsigned)std::min<size_t>((n4 + 255) / 256, (size_t)sm_count() * 8);
    TraceScope trace("scan_step_kernel", s);
    if (a.bf16)
        scan_step_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
            (const __nv_bfloat16*)a.x, a.log_a, a.h0, (__nv_bfloat16*)a.h, a.h_out, n4);
    else
        scan_step_kernel<float><<<grid, 256, 0, s>>>((const float*)a.x, a.log_a, a.h0, (float*)a.h,
                                                     a.h_out, n4);
    return cudaGetLastError();
}

}  // namespace la
