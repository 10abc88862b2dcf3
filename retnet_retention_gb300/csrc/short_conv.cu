// The short causal convolution over each channel of [B][T][D],
//
//   u_t = bias + sum_j w[c][j] x_(t-W+1+j),   y = u  or  u sigmoid(u),
//
// the W - 1 rows before the first token from a state; a tap k tokens back counts only
// where k <= positions[t], by a selection, so that what lies before a document's first
// token does not pass.  Its gradients (du = dy act'(u), recomputed from x):
//
//   dx_s = sum_k w[c][W-1-k] du_(s+k),  dw[c][W-1-k] = sum_t du_t x_(t-k),  dbias = sum du
//
// and its single step.
//
// Bound by HBM: x in, y out, 2 W + 6 operations an entry.  A thread keeps a vector of
// channels (16 bytes; backward four) and walks a run of tokens with the last W - 1 rows
// in registers, so that x is read once but for the W - 1 rows before a run (and backward
// behind it); the loads of the next rows are in flight meanwhile.
#include <algorithm>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kThreads = 128;

// V neighbouring entries as they lie in memory, and as fp32.
template <typename T, int V>
struct Pack {
    static constexpr int kWords = V * (int)sizeof(T) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kWords == 4) {
            const uint4 r = *reinterpret_cast<const uint4*>(p);
            w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
        } else {
            const uint2 r = *reinterpret_cast<const uint2*>(p);
            w[0] = r.x; w[1] = r.y;
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kWords == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void floats(float (&x)[V]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void round(const float (&x)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = bf16x2_bits(x[2 * i], x[2 * i + 1]);
        }
    }
};

struct ConvParams {
    const void *x, *dy;
    long long xb, xt, yb, yt, gb, gt, db, dt;  // strides of x, y, dy, dx: batch, token
    const float *w, *bias;                     // bias may be null
    const void *state, *dstate_T;              // [B][W-1][D] or null
    const int* positions;                      // or null
    void *y, *state_out;                       // forward; state_out may be null
    void *dx, *dstate;                         // backward; dstate may be null
    float *part_w, *part_b;                    // backward: a row for each block of runs, or null
    int B, T, D, silu;
    int lanes;                                 // threads of a CTA side by side on a row
    int tiles;                                 // CTAs side by side
    int run;                                   // tokens of a run
    long long runs;                            // of all sequences
    int runs_per_seq;
    long long run_blocks;                      // CTAs below one another (backward: they stride)
};

// The W weights of V channels from c on.
template <int W, int V>
__device__ __forceinline__ void load_weights(const ConvParams& p, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = __ldg(p.w + (size_t)(c + i) * W + j);
        bias[i] = p.bias ? __ldg(p.bias + c + i) : 0.f;
    }
}

// Row `at` (below 0: of the state) of sequence b.
template <typename T, int W, int V>
__device__ __forceinline__ void row_before(const ConvParams& p, long long b, int at, int c, float (&x)[V]) {
    Pack<T, V> r;
    r.zero();
    if (at >= 0) r.load((const T*)p.x + b * p.xb + at * p.xt + c);
    else if (p.state) r.load((const T*)p.state + (b * (W - 1) + at + (W - 1)) * p.D + c);
    r.floats(x);
}

// u of a token whose row is `cur` behind the rows `before` (oldest first).
template <int W, int V>
__device__ __forceinline__ void convolve(const float (&w)[W][V], const float (&bias)[V],
                                         const float (&before)[W - 1][V], const float (&cur)[V], int reach,
                                         float (&u)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = fmaf(w[W - 1][i], cur[i], bias[i]);
    if (reach >= W - 1) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = fmaf(w[j][i], before[j][i], u[i]);
    } else {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            if (W - 1 - j <= reach)
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] = fmaf(w[j][i], before[j][i], u[i]);
    }
}

template <int W, int V>
__device__ __forceinline__ void push_row(float (&before)[W - 1][V], const float (&cur)[V]) {
#pragma unroll
    for (int j = 0; j < W - 2; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) before[j][i] = before[j + 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) before[W - 2][i] = cur[i];
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 4) short_conv_kernel(const __grid_constant__ ConvParams p) {
    constexpr int V = 16 / (int)sizeof(T), kAhead = 8;  // rows whose loads are in flight
    const int tile = (int)(blockIdx.x % (unsigned)p.tiles);
    const int c = (tile * p.lanes + (int)threadIdx.x % p.lanes) * V;
    const long long run = (long long)(blockIdx.x / (unsigned)p.tiles) * (kThreads / p.lanes) + threadIdx.x / p.lanes;
    if (c >= p.D || run >= p.runs) return;
    const long long b = run / p.runs_per_seq;
    const int t0 = (int)(run - b * p.runs_per_seq) * p.run, t1 = (int)min((long long)t0 + p.run, (long long)p.T);
    float w[W][V], bias[V], before[W - 1][V];
    load_weights<W, V>(p, c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row_before<T, W, V>(p, b, t0 - (W - 1) + j, c, before[j]);
    if (t0 == 0 && p.state_out) {
        // the sequence's first thread has read the state and may write it in place: row j
        // is row T - W + 1 + j of the tokens behind it
        float last[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) row_before<T, W, V>(p, b, p.T - (W - 1) + j, c, last[j]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            Pack<T, V> r;
            r.round(last[j]);  // exact: they are T's
            r.store((T*)p.state_out + (b * (W - 1) + j) * p.D + c);
        }
    }
    const T* x = (const T*)p.x + b * p.xb + (long long)t0 * p.xt + c;
    T* y = (T*)p.y + b * p.yb + (long long)t0 * p.yt + c;
    const int* pos = p.positions ? p.positions + b * p.T + t0 : nullptr;
    const int n = t1 - t0;
    Pack<T, V> next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < n) next[i].load(x + i * p.xt);
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        x += kAhead * p.xt;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i0 + i < n) {
                float cur[V], u[V];
                next[i].floats(cur);
                if (i0 + i + kAhead < n) next[i].load(x + i * p.xt);
                convolve<W, V>(w, bias, before, cur, pos ? __ldg(pos + i0 + i) : W - 1, u);
                push_row<W, V>(before, cur);
                if (p.silu) {
#pragma unroll
                    for (int k = 0; k < V; ++k) u[k] *= sigmoid<T>(u[k]);
                }
                Pack<T, V> r;
                r.round(u);
                r.store(y);
                y += p.yt;
            }
        }
    }
}

// A thread walks its runs forward: at token t it knows u_t and du_t, which complete dx of
// token t - W + 1.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 4) short_conv_bwd_kernel(const __grid_constant__ ConvParams p) {
    constexpr int V = 4, kAhead = 4;
    tc::griddep_launch_dependents();  // the sums' kernel may be scheduled (it waits itself)
    __shared__ float red[kThreads][V + 1];
    const int tile = (int)(blockIdx.x % (unsigned)p.tiles), lane = (int)threadIdx.x % p.lanes;
    const int c = (tile * p.lanes + lane) * V, depth = kThreads / p.lanes, row = (int)threadIdx.x / p.lanes;
    const long long run_block = blockIdx.x / (unsigned)p.tiles;
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    if (c < p.D) {
        float w[W][V], bias[V];
        load_weights<W, V>(p, c, w, bias);
        for (long long run = run_block * depth + row; run < p.runs; run += p.run_blocks * depth) {
            const long long b = run / p.runs_per_seq;
            const int t0 = (int)(run - b * p.runs_per_seq) * p.run;
            const int t1 = (int)min((long long)t0 + p.run, (long long)p.T), n = t1 - t0;
            const int there = min(p.T - t0, n + W - 1);  // tokens to read
            float before[W - 1][V], acc[W][V];           // acc[k]: dx of token t - k so far
#pragma unroll
            for (int j = 0; j < W - 1; ++j) row_before<T, W, V>(p, b, t0 - (W - 1) + j, c, before[j]);
#pragma unroll
            for (int k = 0; k < W; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
            const T* x = (const T*)p.x + b * p.xb + (long long)t0 * p.xt + c;
            const T* dy = (const T*)p.dy + b * p.gb + (long long)t0 * p.gt + c;
            T* dx = (T*)p.dx + b * p.db + (long long)t0 * p.dt + c;
            const int* pos = p.positions ? p.positions + b * p.T + t0 : nullptr;
            Pack<T, V> next_x[kAhead], next_dy[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (i < there) {
                    next_x[i].load(x + i * p.xt);
                    next_dy[i].load(dy + i * p.gt);
                }
            for (int i0 = 0; i0 < n + W - 1; i0 += kAhead) {
                x += kAhead * p.xt;
                dy += kAhead * p.gt;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int m = i0 + i;  // token t0 + m
                    if (m < there) {
                        float cur[V], du[V];
                        next_x[i].floats(cur);
                        next_dy[i].floats(du);
                        if (m + kAhead < there) {
                            next_x[i].load(x + i * p.xt);
                            next_dy[i].load(dy + i * p.gt);
                        }
                        const int reach = pos ? __ldg(pos + m) : W - 1;
                        if (p.silu) {
                            float u[V];
                            convolve<W, V>(w, bias, before, cur, reach, u);
#pragma unroll
                            for (int k = 0; k < V; ++k) {
                                const float s = sigmoid<T>(u[k]), a = u[k] * s;
                                du[k] *= fmaf(a, 1.f - s, s);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < W; ++k) {
                            if (k == 0 || k <= reach) {
#pragma unroll
                                for (int e = 0; e < V; ++e) {
                                    acc[k][e] = fmaf(w[W - 1 - k][e], du[e], acc[k][e]);
                                    const float at = k == 0 ? cur[e] : before[k == 0 ? 0 : W - 1 - k][e];
                                    if (m < n) dw[W - 1 - k][e] = fmaf(du[e], at, dw[W - 1 - k][e]);
                                }
                            }
                        }
                        if (m < n) {
#pragma unroll
                            for (int e = 0; e < V; ++e) db[e] += du[e];
                        }
                        push_row<W, V>(before, cur);
                    }
                    const int s = m - (W - 1);  // token t0 + s has its whole sum
                    if (s < n && (s >= 0 || t0 == 0)) {
                        const int t = t0 + s, k = t - (p.T - (W - 1));
                        if (p.dstate_T && k >= 0) {
                            Pack<T, V> r;
                            float tail[V];
                            r.load((const T*)p.dstate_T + (b * (W - 1) + k) * p.D + c);
                            r.floats(tail);
#pragma unroll
                            for (int e = 0; e < V; ++e) acc[W - 1][e] += tail[e];
                        }
                        Pack<T, V> r;
                        r.round(acc[W - 1]);
                        if (s >= 0) r.store(dx + s * p.dt);
                        else if (p.dstate) r.store((T*)p.dstate + (b * (W - 1) + m) * p.D + c);
                    }
#pragma unroll
                    for (int k = W - 1; k > 0; --k)
#pragma unroll
                        for (int e = 0; e < V; ++e) acc[k][e] = acc[k - 1][e];
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[0][e] = 0.f;
                }
            }
        }
    }
    // one partial row a block of runs: over the CTA's threads of the same channels
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float* part = j < W ? p.part_w : p.part_b;
        if (!part) continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) red[threadIdx.x][e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        if (row == 0 && c < p.D) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float sum = 0.f;
                for (int r = 0; r < depth; ++r) sum += red[r * p.lanes + lane][e];
                if (j < W) part[(size_t)run_block * p.D * W + (size_t)(c + e) * W + j] = sum;
                else part[(size_t)run_block * p.D + c + e] = sum;
            }
        }
    }
}

// One token of each sequence: the state's rows move up by one.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const __grid_constant__ ConvParams p, unsigned vectors) {
    constexpr int V = 16 / (int)sizeof(T);
    const unsigned i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= vectors) return;
    const unsigned per = (unsigned)p.D / V;
    const long long b = i / per;
    const int c = (int)(i - (unsigned)b * per) * V;
    Pack<T, V> rows[W], out;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[j].load((const T*)p.state + (b * (W - 1) + j) * p.D + c);
    rows[W - 1].load((const T*)p.x + b * p.xb + c);
    float w[W][V], u[V];
    load_weights<W, V>(p, c, w, u);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[j + 1].store((T*)p.state_out + (b * (W - 1) + j) * p.D + c);
    float x[V];
    rows[W - 1].floats(x);
#pragma unroll
    for (int k = 0; k < V; ++k) u[k] = fmaf(w[W - 1][k], x[k], u[k]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        rows[j].floats(x);
#pragma unroll
        for (int k = 0; k < V; ++k) u[k] = fmaf(w[j][k], x[k], u[k]);
    }
    if (p.silu) {
#pragma unroll
        for (int k = 0; k < V; ++k) u[k] *= sigmoid<T>(u[k]);
    }
    out.round(u);
    out.store((T*)p.y + b * p.D + c);
}

ConvParams params(const ShortConvArgs& a) {
    ConvParams p = {};
    p.x = a.x; p.dy = a.dy;
    p.xb = a.x_strides[0]; p.xt = a.x_strides[1];
    p.yb = a.y_strides[0]; p.yt = a.y_strides[1];
    p.gb = a.dy_strides[0]; p.gt = a.dy_strides[1];
    p.db = a.dx_strides[0]; p.dt = a.dx_strides[1];
    p.w = a.weight; p.bias = a.bias;
    p.state = a.state; p.dstate_T = a.dstate_T;
    p.positions = a.positions;
    p.y = a.y; p.state_out = a.state_out;
    p.dx = a.dx; p.dstate = a.dstate;
    p.B = a.B; p.T = a.T; p.D = a.D; p.silu = a.silu;
    return p;
}

// Tiles of up to 32 vectors of V channels; runs of `most` tokens where that leaves
// `waves` CTAs a place, shorter ones (down to 8) where it does not.
void shape(ConvParams* p, int V, int most, int waves) {
    const int vectors = p->D / V;
    p->lanes = 32;
    while (p->lanes / 2 >= vectors) p->lanes /= 2;
    p->tiles = (vectors + p->lanes - 1) / p->lanes;
    const long long want = (long long)sm_count() * 4 * waves * (kThreads / p->lanes);  // runs, of all tiles
    const long long tokens = (long long)p->B * p->T * p->tiles;
    long long run = std::min<long long>(std::max<long long>(tokens / want / 8 * 8, 8), most);
    p->run = (int)run;
    p->runs_per_seq = (int)((p->T + run - 1) / run);
    p->runs = (long long)p->B * p->runs_per_seq;
    p->run_blocks = (p->runs + kThreads / p->lanes - 1) / (kThreads / p->lanes);
}

constexpr int kFwdRun = 64, kBwdRun = 64, kBwdBlocksPerSm = 4;

ConvParams bwd_params(const ShortConvArgs& a) {
    ConvParams p = params(a);
    shape(&p, 4, kBwdRun, 1);
    const long long most = ((long long)sm_count() * kBwdBlocksPerSm + p.tiles - 1) / p.tiles;
    p.run_blocks = std::min(p.run_blocks, most);
    return p;
}

template <typename F>
cudaError_t by_width(int W, const F& f) {
    switch (W) {
        case 2: f(std::integral_constant<int, 2>()); break;
        case 3: f(std::integral_constant<int, 3>()); break;
        default: f(std::integral_constant<int, 4>()); break;
    }
    return cudaGetLastError();
}

}  // namespace

size_t short_conv_bwd_workspace_bytes(const ShortConvArgs& a) {
    return (size_t)bwd_params(a).run_blocks * a.D * (a.W + 1) * sizeof(float);
}

cudaError_t launch_short_conv_fwd(const ShortConvArgs& a, cudaStream_t s) {
    ConvParams p = params(a);
    shape(&p, a.bf16 ? 8 : 4, kFwdRun, 4);
    const dim3 grid((unsigned)(p.run_blocks * p.tiles));
    TraceScope trace("short_conv_kernel", s);
    return by_width(a.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        if (a.bf16) short_conv_kernel<__nv_bfloat16, W><<<grid, kThreads, 0, s>>>(p);
        else short_conv_kernel<float, W><<<grid, kThreads, 0, s>>>(p);
    });
}

cudaError_t launch_short_conv_bwd(const ShortConvArgs& a, cudaStream_t s) {
    ConvParams p = bwd_params(a);
    if (a.dweight) p.part_w = (float*)a.workspace;
    if (a.dbias) p.part_b = (float*)a.workspace + (size_t)p.run_blocks * a.D * a.W;
    const dim3 grid((unsigned)(p.run_blocks * p.tiles));
    cudaError_t e;
    {
        TraceScope trace("short_conv_bwd_kernel", s);
        e = by_width(a.W, [&](auto w) {
            constexpr int W = decltype(w)::value;
            if (a.bf16) short_conv_bwd_kernel<__nv_bfloat16, W><<<grid, kThreads, 0, s>>>(p);
            else short_conv_bwd_kernel<float, W><<<grid, kThreads, 0, s>>>(p);
        });
    }
    if (e != cudaSuccess) return e;
    const PartialSum sums[2] = {{p.part_w, a.dweight, (int)p.run_blocks, a.D * a.W},
                                {p.part_b, a.dbias, (int)p.run_blocks, a.D}};
    return launch_partial_sums(sums, 2, s);
}

cudaError_t launch_short_conv_step(const ShortConvArgs& a, cudaStream_t s) {
    ConvParams p = params(a);
    const unsigned vectors = (unsigned)((long long)a.B * a.D / (a.bf16 ? 8 : 4));
    const unsigned grid = (vectors + kThreads - 1) / kThreads;
    TraceScope trace("short_conv_step_kernel", s);
    return by_width(a.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        if (a.bf16) short_conv_step_kernel<__nv_bfloat16, W><<<grid, kThreads, 0, s>>>(p, vectors);
        else short_conv_step_kernel<float, W><<<grid, kThreads, 0, s>>>(p, vectors);
    });
}

}  // namespace la
