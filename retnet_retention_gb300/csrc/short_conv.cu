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
// behind it).  The next eight rows come through a ring in shared memory, each thread's own
// pieces, copied in the background: loads in flight cost no registers and there is no barrier.
//
// 8 x 8192 tokens of 4096 channels in bf16: 168 us, 6.4 TB/s, 0.95 of the copy rate.  The gradients
// (4 x 4093 tokens of 4096 channels: 92 us, 4.4 TB/s) are bound by their instructions, 112 for a token of
// a warp's 128 channels, 38 of them packed and two turns long; a ring of W - 1 rows in registers beside the
// token's own took 10 more, to move them (96 us); eight channels a thread did not fit the registers (182 us).
// A step of 256 sequences of 4096 channels takes 4.8 us in a graph.
#include <algorithm>
#include <type_traits>

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
    __device__ __forceinline__ void floats(float2 (&x)[V / 2]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (sizeof(T) == 4) x[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
            else x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        }
    }
    __device__ __forceinline__ void round(const float2 (&x)[V / 2]) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[2 * i] = __float_as_uint(x[i].x);
                w[2 * i + 1] = __float_as_uint(x[i].y);
            } else {
                w[i] = bf16x2_bits(x[i].x, x[i].y);
            }
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

// The W weights of V channels from c on (V W neighbouring numbers, V a multiple of 4), as
// pairs of channels for the packed arithmetic.
template <int W, int V>
__device__ __forceinline__ void load_weights(const ConvParams& p, int c, float2 (&w)[W][V / 2], float2 (&bias)[V / 2]) {
    float all[V * W];
#pragma unroll
    for (int i = 0; i < V * W; i += 4)
        *reinterpret_cast<float4*>(all + i) = __ldg(reinterpret_cast<const float4*>(p.w + (size_t)c * W + i));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = make_float2(all[2 * i * W + j], all[(2 * i + 1) * W + j]);
        bias[i] = p.bias ? __ldg(reinterpret_cast<const float2*>(p.bias + c) + i) : make_float2(0.f, 0.f);
    }
}

// Row `at` (below 0: of the state) of sequence b.
template <typename T, int W, int V>
__device__ __forceinline__ Pack<T, V> row_before(const ConvParams& p, long long b, int at, int c) {
    Pack<T, V> r;
    r.zero();
    if (at >= 0) r.load((const T*)p.x + b * p.xb + at * p.xt + c);
    else if (p.state) r.load((const T*)p.state + (b * (W - 1) + at + (W - 1)) * p.D + c);
    return r;
}

// u of a token from the last W rows, its own at rows[AT]: row k back is rows[(AT - k) mod W], a
// place known when the loop is unrolled, so that the rows never move.
template <int W, int V, int AT>
__device__ __forceinline__ void convolve(const float2 (&w)[W][V / 2], const float2 (&bias)[V / 2],
                                         const float2 (&rows)[W][V / 2], int reach, float2 (&u)[V / 2]) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) u[i] = __ffma2_rn(w[W - 1][i], rows[AT][i], bias[i]);
#pragma unroll
    for (int k = W - 1; k > 0; --k) {
        if (k <= reach) {
            constexpr int kWrap = AT + W;
            const int at = (kWrap - k) % W;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) u[i] = __ffma2_rn(w[W - 1 - k][i], rows[at][i], u[i]);
        }
    }
}

// Tokens of the unrolled loop, a multiple of the W rows kept (a long loop does not stay in the
// instruction cache: nine tokens of the gradients took 119 us where three took 96, four 92), and rows of the
// ring, a multiple of those.
template <int W>
constexpr int kUnrollOf = W == 3 ? 3 : 4;
template <int W>
constexpr int kAheadOf = W == 3 ? 9 : 8;

// How far the taps of the next tokens reach, loaded a turn of the loop before it is looked at.
template <int W>
struct Reaches {
    static constexpr int U = kUnrollOf<W>;
    int next[U], now[U];
    bool full;  // all of now's taps count

    __device__ __forceinline__ void load(const int* pos, int m0, int n) {
#pragma unroll
        for (int i = 0; i < U; ++i) next[i] = pos && m0 + i < n ? __ldg(pos + m0 + i) : W - 1;
    }
    __device__ __forceinline__ void turn() {
        full = true;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            now[i] = next[i];
            full = full && now[i] >= W - 1;
        }
    }
};

// f(0), .. f(N - 1) with the index a constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(const F& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        each<N, I + 1>(f);
    }
}

// A thread's V entries from global to shared memory in the background.
template <typename T, int V>
__device__ __forceinline__ void copy_pack(void* to, const T* from) {
    constexpr int kBytes = V * (int)sizeof(T);
    if constexpr (kBytes == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                     : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                     "n"(kBytes)
                     : "memory");
    }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 4) short_conv_kernel(const __grid_constant__ ConvParams p) {
    constexpr int V = 16 / (int)sizeof(T), kAhead = kAheadOf<W>, U = kUnrollOf<W>;
    __shared__ __align__(16) uint4 ring[kAhead][kThreads];
    const int tile = (int)(blockIdx.x % (unsigned)p.tiles);
    const int c = (tile * p.lanes + (int)threadIdx.x % p.lanes) * V;
    const long long run = (long long)(blockIdx.x / (unsigned)p.tiles) * (kThreads / p.lanes) + threadIdx.x / p.lanes;
    if (c >= p.D || run >= p.runs) return;
    const long long b = run / p.runs_per_seq;
    const int t0 = (int)(run - b * p.runs_per_seq) * p.run, t1 = (int)min((long long)t0 + p.run, (long long)p.T);
    const int n = t1 - t0;
    const T* ahead = (const T*)p.x + b * p.xb + (long long)t0 * p.xt + c;
    T* y = (T*)p.y + b * p.yb + (long long)t0 * p.yt + c;
    const int* pos = p.positions ? p.positions + b * p.T + t0 : nullptr;
    auto fetch = [&](int m, int slot) {
        if (m < n) copy_pack<T, V>(&ring[slot][threadIdx.x], ahead);
        copies_commit();
        ahead += p.xt;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i, i);
    float2 w[W][V / 2], bias[V / 2], rows[W][V / 2];  // the token's and those before it
    load_weights<W, V>(p, c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row_before<T, W, V>(p, b, t0 - (W - 1) + j, c).floats(rows[j + 1]);
    if (t0 == 0 && p.state_out) {
        // the sequence's first thread has read the state and may write it in place: row j
        // is row T - W + 1 + j of the tokens behind it
        Pack<T, V> last[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j] = row_before<T, W, V>(p, b, p.T - (W - 1) + j, c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j].store((T*)p.state_out + (b * (W - 1) + j) * p.D + c);
    }
    Reaches<W> reaches;
    reaches.load(pos, 0, n);
    for (int i0 = 0, slot = 0; i0 < n; i0 += U, slot = slot + U == kAhead ? 0 : slot + U) {
        reaches.turn();
        reaches.load(pos, i0 + U, n);
        auto token = [&](auto index, int reach) {
            constexpr int i = decltype(index)::value;
            copies_wait<kAhead - 1>();
            Pack<T, V> r;
            float2 u[V / 2];
            r.load(reinterpret_cast<const T*>(&ring[slot + i][threadIdx.x]));
            r.floats(rows[i % W]);
            fetch(i0 + i + kAhead, slot + i);
            convolve<W, V, i % W>(w, bias, rows, reach, u);
            if (p.silu) {
#pragma unroll
                for (int k = 0; k < V / 2; ++k) u[k] = __fmul2_rn(u[k], sigmoid2<T>(u[k]));
            }
            r.round(u);
            r.store(y);
            y += p.yt;
        };
        if (reaches.full && i0 + U <= n) {
            each<U>([&](auto index) { token(index, W - 1); });
        } else {
            each<U>([&](auto index) {
                constexpr int i = decltype(index)::value;
                if (i0 + i < n) token(index, reaches.now[i]);
            });
        }
    }
}

// A thread walks its runs forward: at token t it knows u_t and du_t, which complete dx of
// token t - W + 1.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 4) short_conv_bwd_kernel(const __grid_constant__ ConvParams p) {
    constexpr int V = 4, kAhead = kAheadOf<W>, U = kUnrollOf<W>;
    tc::griddep_launch_dependents();  // the sums' kernel may be scheduled (it waits itself)
    using Piece = std::conditional_t<sizeof(T) == 2, uint2, uint4>;
    __shared__ __align__(16) Piece ring[kAhead][2][kThreads];  // x, dy
    const int tile = (int)(blockIdx.x % (unsigned)p.tiles), lane = (int)threadIdx.x % p.lanes;
    const int c = (tile * p.lanes + lane) * V, depth = kThreads / p.lanes, row = (int)threadIdx.x / p.lanes;
    const long long run_block = blockIdx.x / (unsigned)p.tiles;
    float2 dw[W][V / 2], db[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        db[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = make_float2(0.f, 0.f);
    }
    if (c < p.D) {
        float2 w[W][V / 2], bias[V / 2];
        load_weights<W, V>(p, c, w, bias);
        for (long long run = run_block * depth + row; run < p.runs; run += p.run_blocks * depth) {
            const long long b = run / p.runs_per_seq;
            const int t0 = (int)(run - b * p.runs_per_seq) * p.run;
            const int t1 = (int)min((long long)t0 + p.run, (long long)p.T), n = t1 - t0;
            const int there = min(p.T - t0, n + W - 1);  // tokens to read
            const T* x = (const T*)p.x + b * p.xb + (long long)t0 * p.xt + c;
            const T* dy = (const T*)p.dy + b * p.gb + (long long)t0 * p.gt + c;
            T* dx = (T*)p.dx + b * p.db + (long long)t0 * p.dt + c;
            const int* pos = p.positions ? p.positions + b * p.T + t0 : nullptr;
            auto fetch = [&](int m, int slot) {
                if (m < there) {
                    copy_pack<T, V>(&ring[slot][0][threadIdx.x], x);
                    copy_pack<T, V>(&ring[slot][1][threadIdx.x], dy);
                }
                copies_commit();
                x += p.xt;
                dy += p.gt;
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i, i);
            float2 rows[W][V / 2], dus[W][V / 2];  // the token's row and the last ones, their du
            int reached[W];                        // and, where not all, how far their taps reached
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (j > 0) row_before<T, W, V>(p, b, t0 - W + j, c).floats(rows[j]);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) dus[j][e] = make_float2(0.f, 0.f);
            }
            Reaches<W> reaches;
            reaches.load(pos, 0, there);
            bool clean = true;  // the last rows' taps all counted
            for (int i0 = 0, slot = 0; i0 < n + W - 1; i0 += U, slot = slot + U == kAhead ? 0 : slot + U) {
                reaches.turn();
                reaches.load(pos, i0 + U, there);
                // WHOLE: a token of the run, as is the one it completes, every tap counts, and the
                // sequence's last rows are not reached
                auto token = [&](auto index, auto whole) {
                    constexpr int i = decltype(index)::value;
                    constexpr bool kWhole = decltype(whole)::value;
                    const int m = i0 + i;  // token t0 + m
                    constexpr int kAt = i % W;
                    float2(&cur)[V / 2] = rows[kAt], (&du)[V / 2] = dus[kAt];
                    int reach = W - 1;
                    copies_wait<kAhead - 1>();
                    if (!kWhole) {
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) cur[e] = du[e] = make_float2(0.f, 0.f);
                    }
                    if (kWhole || m < there) {
                        Pack<T, V> in;
                        in.load(reinterpret_cast<const T*>(&ring[slot + i][0][threadIdx.x]));
                        in.floats(cur);
                        in.load(reinterpret_cast<const T*>(&ring[slot + i][1][threadIdx.x]));
                        in.floats(du);
                        if (!kWhole) reach = reaches.now[i];
                    }
                    fetch(m + kAhead, slot + i);
                    if (p.silu && (kWhole || m < there)) {
                        float2 u[V / 2];
                        convolve<W, V, kAt>(w, bias, rows, reach, u);
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) {
                            // the slope: sigma + u sigma (1 - sigma)
                            const float2 s = sigmoid2<T>(u[e]), a = __fmul2_rn(u[e], s);
                            du[e] = __fmul2_rn(du[e], __ffma2_rn(a, __ffma2_rn(s, both(-1.f), both(1.f)), s));
                        }
                    }
                    if (kWhole || m < n) {
#pragma unroll
                        for (int k = 0; k < W; ++k) {
                            if (kWhole || k == 0 || k <= reach) {
                                const int from = (kAt + W - k) % W;
#pragma unroll
                                for (int e = 0; e < V / 2; ++e)
                                    dw[W - 1 - k][e] = __ffma2_rn(du[e], rows[from][e], dw[W - 1 - k][e]);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) db[e] = __fadd2_rn(db[e], du[e]);
                    }
                    const int s = m - (W - 1);  // token t0 + s has its whole sum
                    if (kWhole || (s < n && (s >= 0 || t0 == 0))) {
                        float2 sum[V / 2];
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) sum[e] = make_float2(0.f, 0.f);
                        const int t = t0 + s, k_last = t - (p.T - (W - 1));
                        if (!kWhole && p.dstate_T && k_last >= 0) {
                            Pack<T, V> r;
                            r.load((const T*)p.dstate_T + (b * (W - 1) + k_last) * p.D + c);
                            r.floats(sum);
                        }
#pragma unroll
                        for (int k = 0; k < W; ++k) {  // du of token s + k, which lies W - 1 - k back
                            const int from = (kAt + k + 1) % W;
                            const int far = k == W - 1 ? reach : reached[from];
                            if (kWhole || k == 0 || far >= k) {
#pragma unroll
                                for (int e = 0; e < V / 2; ++e)
                                    sum[e] = __ffma2_rn(w[W - 1 - k][e], dus[from][e], sum[e]);
                            }
                        }
                        Pack<T, V> r;
                        r.round(sum);
                        if (kWhole || s >= 0) r.store(dx);
                        else if (p.dstate) r.store((T*)p.dstate + (b * (W - 1) + m) * p.D + c);
                    }
                    if (kWhole || s >= 0) dx += p.dt;
                    if (!kWhole) reached[kAt] = reach;
                };
                if (reaches.full && clean && i0 >= W - 1 && i0 + U <= n) {
                    each<U>([&](auto index) { token(index, std::true_type()); });
                } else {
                    if (clean) {
#pragma unroll
                        for (int j = 0; j < W; ++j) reached[j] = W - 1;
                    }
                    each<U>([&](auto index) {
                        if (i0 + decltype(index)::value < n + W - 1) token(index, std::false_type());
                    });
                }
                clean = reaches.full;  // U is at least W - 1
            }
            copies_wait<0>();
        }
    }
    // one partial row a block of runs: over the CTA's threads of the same channels
    float2(*red)[V / 2] = reinterpret_cast<float2(*)[V / 2]>(&ring[0][0][0]);
    static_assert(sizeof(ring) >= kThreads * V * sizeof(float), "a thread's sums of one tap fit the ring");
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float* part = j < W ? p.part_w : p.part_b;
        if (!part) continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V / 2; ++e) red[threadIdx.x][e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        if (row == 0 && c < p.D) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float sum = 0.f;
                for (int r = 0; r < depth; ++r) {
                    const float2 v = red[r * p.lanes + lane][e / 2];
                    sum += e % 2 ? v.y : v.x;
                }
                if (j < W) part[(size_t)run_block * p.D * W + (size_t)(c + e) * W + j] = sum;
                else part[(size_t)run_block * p.D + c + e] = sum;
            }
        }
    }
}

// One token of each sequence, with PLACED its taps as far back as its position says: the state's
// rows move up by one.  A thread keeps its channels' weights (as many bytes as a sequence's rows)
// and walks sequences.  Without positions a build of its own: 4.8 us at the size above, where asking
// after them took 4.9.
template <typename T, int W, bool PLACED>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const __grid_constant__ ConvParams p) {
    constexpr int V = 16 / (int)sizeof(T);
    const int c = (int)(blockIdx.x * kThreads + threadIdx.x) * V;
    if (c >= p.D) return;
    Pack<T, V> rows[W], next[W];
    auto load = [&](Pack<T, V>(&to)[W], long long b) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) to[j].load((const T*)p.state + (b * (W - 1) + j) * p.D + c);
        to[W - 1].load((const T*)p.x + b * p.xb + c);
    };
    auto load_reach = [&](long long b) { return PLACED ? __ldg(p.positions + b) : W - 1; };
    load(rows, blockIdx.y);
    int reach = load_reach(blockIdx.y), next_reach = W - 1;
    float2 w[W][V / 2], bias[V / 2];
    load_weights<W, V>(p, c, w, bias);
    for (long long b = blockIdx.y; b < p.B; b += gridDim.y) {
        if (b + gridDim.y < p.B) {
            load(next, b + gridDim.y);
            next_reach = load_reach(b + gridDim.y);
        }
        float2 u[V / 2], x[W][V / 2];
#pragma unroll
        for (int j = 0; j < W; ++j) rows[j].floats(x[j]);
#pragma unroll
        for (int j = 1; j < W; ++j) rows[j].store((T*)p.state_out + (b * (W - 1) + j - 1) * p.D + c);
        convolve<W, V, W - 1>(w, bias, x, reach, u);
        if (p.silu) {
#pragma unroll
            for (int k = 0; k < V / 2; ++k) u[k] = __fmul2_rn(u[k], sigmoid2<T>(u[k]));
        }
        Pack<T, V> out;
        out.round(u);
        out.store((T*)p.y + b * p.D + c);
#pragma unroll
        for (int j = 0; j < W; ++j) rows[j] = next[j];
        reach = next_reach;
    }
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

// Tiles of up to 32 vectors of V channels.
void tile(ConvParams* p, int V) {
    const int vectors = p->D / V;
    p->lanes = 32;
    while (p->lanes / 2 >= vectors) p->lanes /= 2;
    p->tiles = (vectors + p->lanes - 1) / p->lanes;
}

void cut(ConvParams* p, long long run) {
    p->run = (int)run;
    p->runs_per_seq = (int)((p->T + run - 1) / run);
    p->runs = (long long)p->B * p->runs_per_seq;
    const int depth = kThreads / p->lanes;  // runs of a CTA
    p->run_blocks = (p->runs + depth - 1) / depth;
}

constexpr int kRun = 64, kCtasPerSm = 4;

// Forward: runs of kRun tokens where that leaves every SM four times the CTAs it holds,
// shorter ones (down to 8) where it does not.
ConvParams fwd_params(const ShortConvArgs& a) {
    ConvParams p = params(a);
    tile(&p, a.bf16 ? 8 : 4);
    const long long want = (long long)sm_count() * kCtasPerSm * 4 * (kThreads / p.lanes);  // runs, of all tiles
    const long long tokens = (long long)p.B * p.T * p.tiles;
    cut(&p, std::min<long long>(std::max<long long>(tokens / want / 8 * 8, 8), kRun));
    return p;
}

// Backward: the CTAs that fit at once, each as many runs of about kRun tokens as the others (4 x 4093
// tokens of 4096 channels: 228 runs of 72 tokens, three for each of 76 places; with 256 of 64 some
// places would take four).
ConvParams bwd_params(const ShortConvArgs& a) {
    ConvParams p = params(a);
    tile(&p, 4);
    const long long blocks = ((long long)sm_count() * kCtasPerSm + p.tiles - 1) / p.tiles;
    const long long places = blocks * (kThreads / p.lanes), tokens = (long long)p.B * p.T;
    const long long turns = std::max<long long>(1, (tokens + places * kRun / 2) / (places * kRun));
    const long long per_seq = std::max<long long>(1, places * turns / p.B);
    cut(&p, std::max<long long>(8, (p.T + per_seq - 1) / per_seq));
    p.run_blocks = std::min(p.run_blocks, blocks);
    return p;
}

constexpr int kStepBlocksPerSm = 4;

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
    const ConvParams p = fwd_params(a);
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
    const ConvParams p = params(a);
    const int vectors = a.D / (a.bf16 ? 8 : 4);
    const unsigned blocks = (unsigned)((vectors + kThreads - 1) / kThreads);
    const long long want = ((long long)sm_count() * kStepBlocksPerSm + blocks - 1) / blocks;
    const dim3 grid(blocks, (unsigned)std::min<long long>(std::min<long long>(a.B, want), 65535));
    TraceScope trace("short_conv_step_kernel", s);
    return by_width(a.W, [&](auto w) {
        constexpr int W = decltype(w)::value;
        auto step = [&](auto placed) {
            constexpr bool kPlaced = decltype(placed)::value;
            if (a.bf16) short_conv_step_kernel<__nv_bfloat16, W, kPlaced><<<grid, kThreads, 0, s>>>(p);
            else short_conv_step_kernel<float, W, kPlaced><<<grid, kThreads, 0, s>>>(p);
        };
        if (p.positions) step(std::true_type());
        else step(std::false_type());
    });
}

}  // namespace la
