// The selective scan over [B][T][D] with N numbers of state a channel (csrc/ssm.cu,
// csrc/ssm_bwd.cuh): parameters, the elementwise parts and the walk over tokens.
//
//   delta = softplus(dt + dt_bias)  (or the sum itself)
//   h_t = exp(delta A) h_(t-1) + delta x b_t,   y_t = (c_t . h_t + skip x) gate sigmoid(gate)
#pragma once

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

struct SsmRows {
    const void* p;
    long long b, t;  // strides: batch, token
};

struct SsmParams {
    SsmRows x, dt, gate, bm, cm, dy, y;  // gate, dy may be absent (null)
    const float *A, *skip, *bias;        // [D][N]; skip, bias may be null
    const int* positions;                // or null
    const float* h0;                     // [B][D][N] or null
    float* h_out;                        // or null
    // chunks of a sequence: the state entering each, or left by each from none, and the
    // sum of its delta (infinity where a document starts in it)
    float *chunk_h, *chunk_s;            // [B][chunks][D][N], [B][chunks][D]
    float *chunk_g;                      // backward: what each passes back, [B][chunks][D][N]
    // backward: the local state before every kBlock tokens and the sum of delta up to there
    float *block_h, *block_s;            // [B][blocks][D][N], [B][blocks][D]
    int B, T, D, N, G;
    int channels;                        // of a group, D / G
    int tiles;                           // CTAs a group's channels take
    int chunks, chunk;                   // chunks of a sequence, tokens of one
    int blocks;                          // ceil(T / kBlock)
    int softplus;
};

// The gradients' second walk: SsmParams beside what it writes.
struct SsmBwdParams {
    SsmParams f;
    SsmRows dx, ddt, dgate;              // outputs
    float *part_A, *part_skip, *part_bias;  // [B chunks][D][N], [B chunks][D] twice; or null
    float* part_bc;                      // [G tiles][B][T][2 N]
    float* dh0;                          // or null
};

namespace ssm {

constexpr int kBlock = 8;    // tokens a lane group works on at once
constexpr int kTile = 32;    // tokens whose b and c lie in shared memory
constexpr int kWarps = 4;

// 2^v, 2 ulp; 0 below the fp32 range.
__device__ __forceinline__ float exp2_fast(float v) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
    return e;
}

constexpr float kLog2e = 1.4426950408889634f;

// log(1 + p) for p in [0, 1], 1.7e-7 relative (p = 0 included): p times a polynomial of
// degree 8 fitted to log(1 + p) / p in the relative maximum norm.  No logarithm, so that
// small steps keep all their digits.
__device__ __forceinline__ float log1p_unit(float p) {
    float q = 0.00523269409f;
    q = fmaf(q, p, -0.0295052379f);
    q = fmaf(q, p, 0.0782259554f);
    q = fmaf(q, p, -0.136632457f);
    q = fmaf(q, p, 0.191060066f);
    q = fmaf(q, p, -0.24842982f);
    q = fmaf(q, p, 0.333190978f);
    q = fmaf(q, p, -0.499994934f);
    q = fmaf(q, p, 0.99999994f);
    return q * p;
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|); the bf16 form takes 2^x of the scaled
// argument (its error, relative, 2^-22 |v|), fp32 expf.
template <typename T>
__device__ __forceinline__ float softplus(float v) {
    const float p = sizeof(T) == 2 ? exp2_fast(-fabsf(v) * kLog2e) : expf(-fabsf(v));
    return fmaxf(v, 0.f) + log1p_unit(p);
}

template <typename T>
__device__ __forceinline__ float load_one(const T* p) {
    return load_elem(p, 0);
}

// v[0 .. L-1] of the L lanes that lie `gap` apart, lane j keeps the sum of v[j].
template <int L>
__device__ __forceinline__ float share_sums(float (&v)[L], int j, int gap) {
    if constexpr (L > 1) {
#pragma unroll
        for (int s = L / 2; s > 0; s /= 2) {
            const bool hi = j & s;
#pragma unroll
            for (int i = 0; i < s; ++i) {
                const float keep = hi ? v[i + s] : v[i], send = hi ? v[i] : v[i + s];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s * gap);
            }
        }
    }
    return v[0];
}

// The rows of b and c of a tile of tokens, as fp32 [token][2 N]: loads into registers
// ahead of time, then into shared memory.
template <typename T, int N, int THREADS, int TOKENS>
struct SharedRows {
    static constexpr int kPieces = TOKENS * 2 * N / 8, kEach = (kPieces + THREADS - 1) / THREADS;
    Raw8<T> raw[kEach];

    __device__ __forceinline__ void load(const SsmParams& p, long long b, int g, int t0, int t1) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int q = i * THREADS + threadIdx.x, row = q / (2 * N / 8), part = q % (2 * N / 8);
            const bool c = part >= N / 8;
            const SsmRows& from = c ? p.cm : p.bm;
            raw[i] = Raw8<T>();
            if (q < kPieces && t0 + row < t1)
                raw[i] = raw8<true>((const T*)from.p + b * from.b + (long long)(t0 + row) * from.t + g * N +
                                        (part - (c ? N / 8 : 0)) * 8, 0, 4);
        }
    }
    __device__ __forceinline__ void store(float* to) const {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int q = i * THREADS + threadIdx.x;
            if (q < kPieces) {
                float2 x[4];
                floats8<false>(raw[i], x);
                store8<true, false>(to + q * 8, 0, 4, x);
            }
        }
    }
};

enum Mode { kForward, kState, kSummary };  // kState: a chunk's state alone; kSummary: for the gradients

// One walk over a chunk of tokens for a tile of channels.  A channel's N states lie with
// L lanes, NS = N / L each, CW = 32 / L lanes apart; the elementwise work of kBlock tokens is shared
// out to the L lanes token by token.  kForward writes y from the state entering the chunk;
// kState leaves the state the chunk reaches from zero and the sum of delta; kSummary also what
// it passes back, sum_t (prod_(s <= t) e_s) c_t du_t, and the local states every kBlock tokens.
template <typename T, int NS, int L, Mode MODE>
__global__ void __launch_bounds__(kWarps * 32) ssm_scan_kernel(const __grid_constant__ SsmParams p) {
    constexpr int N = NS * L, CW = 32 / L, U = kBlock, K = U / L, kThreads = kWarps * 32;
    constexpr bool kY = MODE == kForward, kBack = MODE == kSummary;
    __shared__ __align__(16) float bc[2][kTile][2 * N];
    __shared__ unsigned starts[2];  // tokens of the tile that start a document
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = lane / CW;
    unsigned unit = blockIdx.x;
    const unsigned tile = unit % (unsigned)(p.tiles * p.G);
    unit /= (unsigned)(p.tiles * p.G);
    const int chunk = (int)(unit % (unsigned)p.chunks);
    const long long b = unit / (unsigned)p.chunks;
    const int g = (int)(tile / (unsigned)p.tiles);
    const int in_group = (int)(tile % (unsigned)p.tiles) * (kWarps * CW) + w * CW + lane % CW;
    const bool on = in_group < p.channels;
    const int c = g * p.channels + (on ? in_group : 0);
    const int t0 = chunk * p.chunk, t1 = (int)min((long long)t0 + p.chunk, (long long)p.T);
    const long long state_at = ((b * p.chunks + chunk) * p.D + c) * N + j * NS;

    float A[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A[i] = __ldg(p.A + (size_t)c * N + j * NS + i) * kLog2e;
        h[i] = 0.f;
    }
    if (MODE == kForward) {
        const float* from = p.chunks > 1 ? p.chunk_h + state_at : p.h0 ? p.h0 + (b * p.D + c) * N + j * NS : nullptr;
        if (from) {
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = from[i];
        }
    }
    float P[kBack ? NS : 1], back[kBack ? NS : 1];
    if (kBack) {
#pragma unroll
        for (int i = 0; i < NS; ++i) P[kBack ? i : 0] = 1.f, back[kBack ? i : 0] = 0.f;
    }
    float sum = 0.f;  // of delta
    bool cut = false;
    const float skip = p.skip ? p.skip[c] : 0.f, bias = p.bias ? p.bias[c] : 0.f;

    // the lane's own tokens of a block: t + k L + j
    const T* x_at = (const T*)p.x.p + b * p.x.b + c;
    const T* dt_at = (const T*)p.dt.p + b * p.dt.b + c;
    const T* gate_at = p.gate.p && MODE != kState ? (const T*)p.gate.p + b * p.gate.b + c : nullptr;
    const T* dy_at = kBack ? (const T*)p.dy.p + b * p.dy.b + c : nullptr;
    T nx[K] = {}, ndt[K] = {}, ngate[K] = {}, ndy[K] = {};
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = t + k * L + j;
            if (on && at < t1) {
                nx[k] = x_at[at * p.x.t];
                ndt[k] = dt_at[at * p.dt.t];
                if (gate_at) ngate[k] = gate_at[at * p.gate.t];
                if (kBack) ndy[k] = dy_at[at * p.dy.t];
            }
        }
    };
    SharedRows<T, N, kThreads, kTile> rows;
    int position = 1;
    auto fetch_tile = [&](int t) {
        rows.load(p, b, g, t, t1);
        if (p.positions && w == 0) position = t + lane < t1 ? p.positions[b * p.T + t + lane] : 1;
    };
    auto store_tile = [&](int buf) {
        rows.store(&bc[buf][0][0]);
        if (w == 0) {
            const unsigned m = __ballot_sync(0xffffffffu, position == 0);
            if (lane == 0) starts[buf] = m;
        }
    };
    fetch_tile(t0);
    fetch(t0);
    store_tile(0);
    __syncthreads();
    int buf = 0;
    for (int tt = t0; tt < t1; tt += kTile, buf ^= 1) {
        if (tt + kTile < t1) fetch_tile(tt + kTile);
        const unsigned tile_starts = starts[buf];
        for (int q = 0; q < kTile && tt + q < t1; q += U) {
            const int t = tt + q;
            if (kBack && t > t0) {  // the local state before this block of the chunk
                const long long at = (b * p.blocks + t / U) * p.D + c;
                if (on) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) p.block_h[at * N + j * NS + i] = h[i];
                    if (j == 0) p.block_s[at] = cut ? INFINITY : sum;
                }
            }
            float xs[K], d[K], dx[K], gate[K], du[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const bool there = on && t + k * L + j < t1;
                xs[k] = there ? load_one(&nx[k]) : 0.f;
                const float v = load_one(&ndt[k]) + bias;
                d[k] = there ? (p.softplus ? softplus<T>(v) : v) : 0.f;
                dx[k] = d[k] * xs[k];
                gate[k] = there && gate_at ? load_one(&ngate[k]) : 0.f;
                du[k] = kBack && there ? load_one(&ndy[k]) : 0.f;
                if (kBack && gate_at) du[k] *= gate[k] * sigmoid<T>(gate[k]);
            }
            fetch(t + U);
            const unsigned block_starts = tile_starts >> q & ((1u << U) - 1);
            float acc[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int from = u % L * CW + lane % CW;
                const float du_ = d[u / L], dxu_ = dx[u / L];
                const float delta = L == 1 ? du_ : __shfl_sync(0xffffffffu, du_, from);
                const float in = L == 1 ? dxu_ : __shfl_sync(0xffffffffu, dxu_, from);
                float dut = 0.f;
                if (kBack) dut = L == 1 ? du[u / L] : __shfl_sync(0xffffffffu, du[u / L], from);
                float bv[NS], cv[NS];
#pragma unroll
                for (int i = 0; i < NS; i += 4) {
                    *reinterpret_cast<float4*>(bv + i) = *reinterpret_cast<const float4*>(&bc[buf][q + u][j * NS + i]);
                    if (MODE != kState)
                        *reinterpret_cast<float4*>(cv + i) =
                            *reinterpret_cast<const float4*>(&bc[buf][q + u][N + j * NS + i]);
                }
                acc[u] = 0.f;
                if (block_starts >> u & 1) {  // the old state is dropped, not multiplied by zero
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        h[i] = in * bv[i];
                        if (kBack) P[kBack ? i : 0] = 0.f;
                    }
                    cut = true;
                } else {
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const float e = exp2_fast(delta * A[i]);
                        h[i] = fmaf(e, h[i], in * bv[i]);
                        if (kBack) P[kBack ? i : 0] *= e;
                    }
                }
                if (kY) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) acc[u] = fmaf(cv[i], h[i], acc[u]);
                } else {
                    sum += delta;
                }
                if (kBack) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const int k = kBack ? i : 0;
                        back[k] = cut ? back[k] : fmaf(P[k], dut * cv[i], back[k]);
                    }
                }
            }
            if (kY) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float v[L];
#pragma unroll
                    for (int i = 0; i < L; ++i) v[i] = acc[k * L + i];
                    float u = fmaf(skip, xs[k], share_sums<L>(v, j, CW));
                    if (gate_at) u *= gate[k] * sigmoid<T>(gate[k]);
                    const int at = t + k * L + j;
                    if (on && at < t1) store_elem((T*)p.y.p + b * p.y.b + at * p.y.t + c, 0, u);
                }
            }
        }
        if (tt + kTile < t1) store_tile(buf ^ 1);
        __syncthreads();
    }
    if (!on) return;
    if (MODE == kForward) {
        if (p.h_out && t1 == p.T) {
#pragma unroll
            for (int i = 0; i < NS; ++i) p.h_out[(b * p.D + c) * N + j * NS + i] = h[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        p.chunk_h[state_at + i] = h[i];
        if (kBack) p.chunk_g[state_at + i] = back[kBack ? i : 0];
    }
    if (j == 0) p.chunk_s[(b * p.chunks + chunk) * p.D + c] = cut ? INFINITY : sum;
}

// ---- host ----------------------------------------------------------------------------

// Launch the walk with `lanes` lanes a channel (N / lanes in {4, 8, 16}).
template <typename T, Mode MODE>
cudaError_t launch_scan(const SsmParams& p, int lanes, unsigned grid, cudaStream_t s);

// The gradients' second walk (csrc/ssm_bwd.cuh).
template <typename T>
cudaError_t launch_gradients(const SsmBwdParams& p, unsigned grid, cudaStream_t s);

inline int channels_cta(int lanes) { return kWarps * (32 / lanes); }

template <typename T, Mode MODE>
cudaError_t launch_scan_here(const SsmParams& p, int lanes, unsigned grid, cudaStream_t s) {
    TraceScope trace(MODE == kForward ? "ssm_kernel" : MODE == kState ? "ssm_state_kernel" : "ssm_summary_kernel", s);
    const int threads = kWarps * 32, ns = p.N / lanes;
#define LA_SSM_CASE(NS, L) \
    if (ns == NS && lanes == L) ssm_scan_kernel<T, NS, L, MODE><<<grid, threads, 0, s>>>(p);
    LA_SSM_CASE(8, 1)
    LA_SSM_CASE(4, 2)
    LA_SSM_CASE(16, 1)
    LA_SSM_CASE(8, 2)
    LA_SSM_CASE(4, 4)
    LA_SSM_CASE(16, 2)
    LA_SSM_CASE(8, 4)
    LA_SSM_CASE(4, 8)
    LA_SSM_CASE(16, 4)
    LA_SSM_CASE(8, 8)
#undef LA_SSM_CASE
    return cudaGetLastError();
}

}  // namespace ssm
}  // namespace la
