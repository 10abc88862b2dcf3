// The selective scan over [B][T][D] with N numbers of state a channel (csrc/ssm.cu,
// csrc/ssm_bwd.cuh): parameters, the elementwise parts and the walk over tokens.
//
//   delta = softplus(dt + dt_bias)  (or the sum itself)
//   h_t = exp(delta A) h_(t-1) + delta x b_t,   y_t = (c_t . h_t + skip x) gate sigmoid(gate)
//
// The walk is bound by issue slots: for a token of a warp's 32 channels of 16 states 92 instructions, 32 of
// them packed products that take two, so 124 of the 161 cycles it takes where every scheduler has two warps
// (16 x 4096 tokens of 2432 channels: 638 us; with one warp each, 8 sequences, 402).  8 x 8192
// tokens of 4096 channels: 1268 us (the 2^x alone 444, HBM 318); there 104 of 152 SMs hold two CTAs and
// the others one, since a sequence's tokens come one after another.  Not kept, at that size: more lanes a
// channel (1615 to 1810 us), products one by one (slower beside the 2^x), loops of 4 or 16 tokens (1681,
// 1630), more CTAs an SM by fewer registers.
#pragma once

#include <type_traits>

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
constexpr int kTile = 16;    // tokens whose rows lie in shared memory
constexpr int kUnroll = 8;   // tokens of the walk's unrolled loop
constexpr int kWarps = 4;

// 2^v, 2 ulp; 0 below the fp32 range.
__device__ __forceinline__ float exp2_fast(float v) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
    return e;
}

constexpr float kLog2e = 1.4426950408889634f;

// What a token's decay raises the argument of its 2^x by.  exp2_fast comes out low by 2e-8 of itself on
// the average of arguments from -0.3 to -0.003 (measured; 0.6e-8 nearer to 0), and a slow decay is
// applied a thousand times: raised, the mean error is below 0.8e-8 there.  2^kRaise is 1.
constexpr float kRaise = 2e-8f;

// 2^(x / 2), finite: what is carried over many tokens is multiplied by it twice, so that a decay past the
// fp32 range, above 2^128 or below 2^-126, meets a small or large number as token by token, and
// 0 stays 0.  Bounded at 2^127.5, it brings every normal number past the range at x = 255.  What is
// not a number stays so.
__device__ __forceinline__ float bounded_exp2(float v) {
    asm("min.NaN.f32 %0, %0, 0f42ff0000;" : "+f"(v));  // 127.5
    return exp2_fast(v);
}
__device__ __forceinline__ float half_decay(float x) { return bounded_exp2(fmaf(0.5f, x, kRaise)); }

// The same of two states' sum A.
__device__ __forceinline__ float2 half_decay2(float sum, float2 A) {
    const float2 x = __ffma2_rn(both(0.5f * sum), A, both(kRaise));
    return make_float2(bounded_exp2(x.x), bounded_exp2(x.y));
}

// 2^x s + b
__device__ __forceinline__ float carry(float x, float s, float b) {
    const float e = half_decay(x);
    return fmaf(e, e * s, b);
}

// log(1 + p) for p in [0, 1], 1.7e-7 relative (p = 0 included): p times a polynomial of
// degree 8 fitted to log(1 + p) / p in the relative maximum norm.  No logarithm, so that
// small steps keep all their digits.
__device__ __forceinline__ float log1p_coefficient(int i) {
    constexpr float k[9] = {0.00523269409f, -0.0295052379f, 0.0782259554f, -0.136632457f, 0.191060066f,
                            -0.24842982f, 0.333190978f, -0.499994934f, 0.99999994f};
    return k[i];
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|), and its slope 1 / (1 + e^-v) where asked for; the
// bf16 form takes 2^x of the scaled argument (its error, relative, 2^-22 |v|), fp32 expf.
template <typename T>
__device__ __forceinline__ float softplus(float v, float* slope = nullptr) {
    const float p = sizeof(T) == 2 ? exp2_fast(-fabsf(v) * kLog2e) : expf(-fabsf(v));
    if (slope) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + p));  // 1 ulp
        *slope = v >= 0.f ? r : p * r;
    }
    float q = log1p_coefficient(0);
#pragma unroll
    for (int i = 1; i < 9; ++i) q = fmaf(q, p, log1p_coefficient(i));
    return fmaf(q, p, fmaxf(v, 0.f));
}

// The same of two values, packed.
template <typename T>
__device__ __forceinline__ float2 softplus2(float2 v, float2* slope = nullptr) {
    float2 p;
    if (sizeof(T) == 2) {
        const float2 s = __fmul2_rn(make_float2(fabsf(v.x), fabsf(v.y)), both(-kLog2e));
        p = make_float2(exp2_fast(s.x), exp2_fast(s.y));
    } else {
        p = make_float2(expf(-fabsf(v.x)), expf(-fabsf(v.y)));
    }
    if (slope) {
        const float2 one = __fadd2_rn(p, both(1.f));
        float2 r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(one.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(one.y));
        const float2 pr = __fmul2_rn(p, r);
        *slope = make_float2(v.x >= 0.f ? r.x : pr.x, v.y >= 0.f ? r.y : pr.y);
    }
    float2 q = both(log1p_coefficient(0));
#pragma unroll
    for (int i = 1; i < 9; ++i) q = __ffma2_rn(q, p, both(log1p_coefficient(i)));
    return __ffma2_rn(q, p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
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

enum Mode { kForward, kState, kSummary };  // kState: a chunk's state alone; kSummary: for the gradients

// A walk's shape: a channel's N states lie with L lanes, NS = N / L each; a lane holds CH
// channels (1 or 2).  A warp has CL = 32 / L lanes side by side along WC = CH CL channels.
template <typename T, int CH_, int NS_, int L_, Mode MODE_>
struct Shape {
    using Elem = T;
    static constexpr int CH = CH_, NS = NS_, L = L_, N = NS * L, CL = 32 / L, WC = CH * CL;
    static constexpr Mode MODE = MODE_;
    static constexpr int M = L / CH, U = M < kUnroll ? kUnroll : M, K = U / M;  // a lane's own tokens: every M-th, K of U
    // the tile's rows of x, dt, gate and dy of a warp's channels in shared memory, in pieces
    static constexpr int kTensors = MODE == kState ? 2 : MODE == kForward ? 3 : 4;
    static constexpr int kPiece = WC * (int)sizeof(T) < 16 ? WC * (int)sizeof(T) : 16, kElems = kPiece / (int)sizeof(T);
    static constexpr int kPieces = kTile * WC / kElems, kEach = (kPieces + 31) / 32;
    static constexpr int kRows = kTile * WC;       // entries of one tensor's tile
    static constexpr int kSharedRows = kTile * 2 * N;  // of b and c
    static constexpr int kSharedPieces = kSharedRows * (int)sizeof(T) / 16;
    static constexpr int kStage = kTensors * kRows + kSharedRows;  // entries of T
    // a warp's two stages, and b and c as fp32 where they are not
    static constexpr size_t kWarpShared =
        2 * (size_t)kStage * sizeof(T) + (sizeof(T) == 4 ? 0 : kSharedRows * sizeof(float));
    static constexpr size_t kShared = kWarps * kWarpShared;
};

// 8 or 16 bytes from global to shared memory in the background, or as many zeros.
template <int BYTES>
__device__ __forceinline__ void copy_piece(void* to, const void* from, bool valid) {
    if constexpr (BYTES == 16) {
        copy16(to, from, valid);
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                     "l"(from), "n"(BYTES), "r"(valid ? BYTES : 0)
                     : "memory");
    }
}

// What a chunk passes back to one state, sum_t exp(A sum_(s <= t) delta_s) c_t du_t, each decay by its
// exponent: where decays grow, their product P leaves the fp32 range although what it meets is 0 or
// small.
template <typename T>
__device__ __noinline__ float passed_back(const SsmParams& p, long long b, int t0, int t1, int c, int g, int n) {
    const float bias = p.bias ? p.bias[c] : 0.f, A = p.A[(size_t)c * p.N + n] * kLog2e;
    float sum = 0.f, back = 0.f;
    for (int t = t0; t < t1; ++t) {
        if (p.positions && p.positions[b * p.T + t] == 0) break;
        auto at = [&](const SsmRows& r, int e) { return load_elem((const T*)r.p + b * r.b + t * r.t, e); };
        const float v = at(p.dt, c) + bias;
        sum += p.softplus ? softplus<T>(v) : v;
        float du = at(p.dy, c);
        if (p.gate.p) {
            const float z = at(p.gate, c);
            du *= z * sigmoid<T>(z);
        }
        back = carry(sum * A, du * at(p.cm, g * p.N + n), back);
    }
    return back;
}

// One walk over a chunk of tokens for a tile of channels: kForward writes y from the state
// entering the chunk; kState leaves the state the chunk reaches from zero and the sum of
// delta; kSummary also what it passes back, sum_t (prod_(s <= t) e_s) c_t du_t, and the
// local states every kBlock tokens.
//
// A warp copies the next tile's rows in the background, those of its channels and b and c (which
// it brings to fp32 itself: 1.5 instructions a token, and no barrier among warps).  The elementwise work
// of a token and channel is done by one lane: register 0 of CH = 2 is the lane's own channel (2 cl + (j & 1)), and its own
// tokens are every M-th.  Tiles in which a document starts or the chunk ends, and for the summary those
// behind a start, take the careful form of the loop.
template <typename S>
__global__ void __launch_bounds__(kWarps * 32, S::MODE == kState ? 4 : 3)
    ssm_scan_kernel(const __grid_constant__ SsmParams p) {
    using T = typename S::Elem;
    constexpr int CH = S::CH, NS = S::NS, N = S::N, CL = S::CL, WC = S::WC, U = S::U, M = S::M, K = S::K;
    constexpr bool kY = S::MODE == kForward, kBack = S::MODE == kSummary, kGate = S::MODE != kState;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = lane / CL, cl = lane % CL;
    const int own = j / CH, mine = CH * cl + j % CH;  // the own tokens' place, the own channel's
    unsigned unit = blockIdx.x;
    const unsigned tile = unit % (unsigned)(p.tiles * p.G);
    unit /= (unsigned)(p.tiles * p.G);
    const int chunk = (int)(unit % (unsigned)p.chunks);
    const long long b = unit / (unsigned)p.chunks;
    const int g = (int)(tile / (unsigned)p.tiles);
    const int first = (int)(tile % (unsigned)p.tiles) * (kWarps * WC) + w * WC;  // the warp's channels in the group
    int c[CH];
    bool on[CH];
#pragma unroll
    for (int q = 0; q < CH; ++q) {
        const int in_group = first + CH * cl + (CH == 1 ? 0 : q ^ (j & 1));
        on[q] = in_group < p.channels;
        c[q] = g * p.channels + (on[q] ? in_group : 0);
    }
    const int t0 = chunk * p.chunk, t1 = (int)min((long long)t0 + p.chunk, (long long)p.T);
    const bool gated = kGate && p.gate.p != nullptr;

    float A[CH][NS], h[CH][NS];
    float P[CH][kBack ? NS : 1], back[CH][kBack ? NS : 1], sum[CH];
    bool cut = false;
#pragma unroll
    for (int q = 0; q < CH; ++q) {
        sum[q] = 0.f;
        const float* from = nullptr;
        if (kY) {
            if (p.chunks > 1) from = p.chunk_h + ((b * p.chunks + chunk) * p.D + c[q]) * N + j * NS;
            else if (p.h0) from = p.h0 + (b * p.D + c[q]) * N + j * NS;
        }
#pragma unroll
        for (int i = 0; i < NS; i += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + (size_t)c[q] * N + j * NS + i));
            const float4 s = from ? *reinterpret_cast<const float4*>(from + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float as[4] = {a.x, a.y, a.z, a.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                A[q][i + k] = as[k] * kLog2e;
                h[q][i + k] = ss[k];
                if (kBack) P[q][kBack ? i + k : 0] = 1.f, back[q][kBack ? i + k : 0] = 0.f;
            }
        }
    }
    const float skip = p.skip ? p.skip[c[0]] : 0.f, bias = p.bias ? p.bias[c[0]] : 0.f;

    T* const stages = reinterpret_cast<T*>(smem + (size_t)w * S::kWarpShared);
    constexpr int kRows = S::kRows;
    // A lane's piece of a tile's first rows, in each tensor: its place from the tile's start in global
    // memory and in shared memory.  A tile that is all there needs no more than its start.
    constexpr int kPerRow = WC / S::kElems, kPass = 32 / kPerRow;       // pieces of a row, rows a pass
    constexpr int kSharedPerRow = 2 * N * (int)sizeof(T) / 16, kSharedPass = 32 / kSharedPerRow;
    const int row = lane / kPerRow, at = lane % kPerRow * S::kElems;
    const long long col = g * p.channels + first + at;
    const long long x_off = row * p.x.t + col, dt_off = row * p.dt.t + col;
    const long long gate_off = gated ? row * p.gate.t + col : 0, dy_off = kBack ? row * p.dy.t + col : 0;
    const int shared_row = lane / kSharedPerRow, shared_part = lane % kSharedPerRow;
    const bool of_c = shared_part >= kSharedPerRow / 2;
    const SsmRows& shared_rows = of_c ? p.cm : p.bm;
    const T* const shared_from = (const T*)shared_rows.p + b * shared_rows.b + shared_row * shared_rows.t + g * N +
                                 shared_part % (kSharedPerRow / 2) * (16 / (int)sizeof(T));
    const long long shared_t = shared_rows.t;
    const bool whole_channels = first + WC <= p.channels;
    const long long y_off = kY ? row * p.y.t + col : 0;
    auto copy_tile = [&](int buf, int t) {
        T* const stage = stages + buf * S::kStage;
        auto copy_rows = [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
            for (int i = 0; i < S::kEach; ++i) {
                if (S::kPieces >= 32 || lane < S::kPieces) {
                    const bool valid = kWhole || (t + i * kPass + row < t1 && first + at < p.channels);
                    auto copy = [&](int k, const SsmRows& r, long long off) {
                        const T* const from = (const T*)r.p + b * r.b + (t + i * kPass) * r.t;
                        copy_piece<S::kPiece>(stage + k * kRows + (i * kPass + row) * WC + at, valid ? from + off : (const T*)r.p,
                                              valid);
                    };
                    copy(0, p.x, x_off);
                    copy(1, p.dt, dt_off);
                    if (gated) copy(2, p.gate, gate_off);
                    if (kBack) copy(3, p.dy, dy_off);
                }
            }
#pragma unroll
            for (int i = 0; i < (S::kSharedPieces + 31) / 32; ++i) {
                if (S::kSharedPieces >= 32 || lane < S::kSharedPieces) {
                    const bool valid = kWhole || t + i * kSharedPass + shared_row < t1;
                    copy16(stage + S::kTensors * kRows + (i * 32 + lane) * (16 / (int)sizeof(T)),
                           valid ? shared_from + (t + i * kSharedPass) * shared_t : (const T*)shared_rows.p, valid);
                }
            }
        };
        if (whole_channels && t + kTile <= t1) copy_rows(std::true_type());
        else copy_rows(std::false_type());
        copies_commit();
    };
    int position = 1;  // of the lane's token of the next tile
    auto load_position = [&](int t) {
        if (p.positions) position = lane < kTile && t + lane < t1 ? p.positions[b * p.T + t + lane] : 1;
    };
    copy_tile(0, t0);
    load_position(t0);
    int buf = 0;
    for (int tt = t0; tt < t1; tt += kTile, buf ^= 1) {
        const unsigned tile_starts = p.positions ? __ballot_sync(0xffffffffu, position == 0) : 0;
        if (tt + kTile < t1) {
            copy_tile(buf ^ 1, tt + kTile);
            load_position(tt + kTile);
        } else {
            copies_commit();
        }
        copies_wait<1>();
        __syncwarp();
        T* const stage = stages + buf * S::kStage;
        const float* bc = reinterpret_cast<const float*>(stage + S::kTensors * kRows);  // [kTile][2 N]
        if constexpr (sizeof(T) == 2) {
            float* const wide = reinterpret_cast<float*>(stages + 2 * S::kStage);
            bc = wide;
#pragma unroll
            for (int i = 0; i < (S::kSharedPieces + 31) / 32; ++i) {
                const int q = i * 32 + lane;
                if (S::kSharedPieces % 32 == 0 || q < S::kSharedPieces) {
                    float2 v[4];
                    floats8<false>(raw8<true>(stage + S::kTensors * kRows + q * 8, 0, 4), v);
                    store8<true, false>(wide + q * 8, 0, 4, v);
                }
            }
            __syncwarp();
        }
        bc += j * NS;
        T* const own_at = stage + own * WC + mine;
        auto walk = [&](auto careful) {
            constexpr bool kCareful = decltype(careful)::value;
#pragma unroll 1
            for (int q0 = 0; q0 < kTile; q0 += U) {
                const int t = tt + q0;
                if (kCareful && t >= t1) break;
                if (kBack && t > t0 && t % kBlock == 0) {  // the local state before this block of the chunk
                    const long long block = b * p.blocks + t / kBlock;
#pragma unroll
                    for (int q = 0; q < CH; ++q)
                        if (on[q]) {
                            const long long at = block * p.D + c[q];
#pragma unroll
                            for (int i = 0; i < NS; i += 4)
                                *reinterpret_cast<float4*>(p.block_h + at * N + j * NS + i) =
                                    make_float4(h[q][i], h[q][i + 1], h[q][i + 2], h[q][i + 3]);
                            if (j == 0) p.block_s[at] = cut ? INFINITY : sum[q];
                        }
                }
                T* const own_rows = own_at + q0 * WC;
                // two own tokens at a time (one, where it is the only one)
                constexpr int kPairs = (K + 1) / 2;
                float2 xs[kPairs], d[kPairs], dx[kPairs], du[kPairs];
                auto own_pair = [&](int tensor, int k) {
                    return make_float2(load_elem(own_rows + tensor * kRows, 2 * k * M * WC),
                                       K == 1 ? 0.f : load_elem(own_rows + tensor * kRows, (2 * k + 1) * M * WC));
                };
                auto silu = [&](int k) {
                    const float2 z = own_pair(2, k);
                    return __fmul2_rn(z, K == 1 ? make_float2(sigmoid<T>(z.x), 0.f) : sigmoid2<T>(z));
                };
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    xs[k] = own_pair(0, k);
                    const float2 v = __fadd2_rn(own_pair(1, k), both(bias));
                    d[k] = !p.softplus ? v : K == 1 ? make_float2(softplus<T>(v.x), 0.f) : softplus2<T>(v);
                    if (kCareful) {
                        if (t + 2 * k * M + own >= t1) d[k].x = 0.f;
                        if (t + (2 * k + 1) * M + own >= t1) d[k].y = 0.f;
                    }
                    dx[k] = __fmul2_rn(d[k], xs[k]);
                    if (kBack) {
                        du[k] = own_pair(3, k);
                        if (gated) du[k] = __fmul2_rn(du[k], silu(k));
                    }
                }
                const unsigned block_starts = kCareful ? tile_starts >> q0 & ((1u << U) - 1) : 0;
                float acc[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float bv[NS], cv[NS];
#pragma unroll
                    for (int i = 0; i < NS; i += 4) {
                        *reinterpret_cast<float4*>(bv + i) = *reinterpret_cast<const float4*>(bc + (q0 + u) * 2 * N + i);
                        if (S::MODE != kState)
                            *reinterpret_cast<float4*>(cv + i) =
                                *reinterpret_cast<const float4*>(bc + (q0 + u) * 2 * N + N + i);
                    }
                    const bool start = kCareful && (block_starts >> u & 1);
                    if (start) cut = true;
                    float a[CH];
#pragma unroll
                    for (int q = 0; q < CH; ++q) {
                        // from the lane whose own token and channel it is
                        const int from = (u % M * CH + (CH == 1 ? 0 : q ^ (j & 1))) * CL + cl;
                        auto get = [&](const float2(&v)[kPairs]) {
                            const float f = u / M % 2 ? v[u / M / 2].y : v[u / M / 2].x;
                            return M == 1 && q == 0 ? f : __shfl_sync(0xffffffffu, f, from);
                        };
                        const float delta = get(d), in = get(dx), dut = kBack ? get(du) : 0.f;
                        float2 part = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < NS; i += 2) {
                            // two states at a time: a packed operation takes two turns to issue, but
                            // less beside the 2^x than two of its halves
                            const float2 x = __ffma2_rn(both(delta), make_float2(A[q][i], A[q][i + 1]), both(kRaise));
                            const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                            const float2 add = __fmul2_rn(both(in), make_float2(bv[i], bv[i + 1]));
                            float2 hh = __ffma2_rn(e, make_float2(h[q][i], h[q][i + 1]), add);
                            if (start) hh = add;  // the old state is dropped, not multiplied by zero
                            h[q][i] = hh.x;
                            h[q][i + 1] = hh.y;
                            if (kY) part = __ffma2_rn(make_float2(cv[i], cv[i + 1]), hh, part);
                            if (kBack) {
                                const int k = kBack ? i : 0, k1 = kBack ? i + 1 : 0;
                                float2 pp = __fmul2_rn(make_float2(P[q][k], P[q][k1]), e);
                                if (kCareful && cut) pp = make_float2(0.f, 0.f);
                                P[q][k] = pp.x, P[q][k1] = pp.y;
                                const float2 old = make_float2(back[q][k], back[q][k1]);
                                float2 bb = __ffma2_rn(pp, __fmul2_rn(both(dut), make_float2(cv[i], cv[i + 1])), old);
                                if (kCareful && cut) bb = old;
                                back[q][k] = bb.x, back[q][k1] = bb.y;
                            }
                        }
                        a[q] = part.x + part.y;
                        if (!kY) sum[q] += delta;
                    }
                    if (kY) acc[u] = CH == 1 ? a[0] : a[0] + __shfl_xor_sync(0xffffffffu, a[CH - 1], CL);
                }
                if (kY) {
                    auto total = [&](int k) {
                        float v[M];
#pragma unroll
                        for (int i = 0; i < M; ++i) v[i] = acc[k * M + i];
                        return share_sums<M>(v, own, CH * CL);
                    };
#pragma unroll
                    for (int k = 0; k < kPairs; ++k) {
                        float2 u = make_float2(total(2 * k), K == 1 ? 0.f : total(K == 1 ? 0 : 2 * k + 1));
                        u = __ffma2_rn(both(skip), xs[k], u);
                        if (gated) u = __fmul2_rn(u, silu(k));
                        store_elem(own_rows, 2 * k * M * WC, u.x);  // in x's place
                        if (K > 1) store_elem(own_rows, (2 * k + 1) * M * WC, u.y);
                    }
                }
            }
        };
        if (tile_starts == 0 && tt + kTile <= t1 && !(kBack && cut)) walk(std::false_type());
        else walk(std::true_type());
        if (kY) {
            __syncwarp();
            auto put_rows = [&](auto whole) {
                constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
                for (int i = 0; i < S::kEach; ++i) {
                    const bool valid = kWhole || (tt + i * kPass + row < t1 && first + at < p.channels);
                    if ((S::kPieces >= 32 || lane < S::kPieces) && valid) {
                        const T* const from = stage + (i * kPass + row) * WC + at;
                        T* const to = (T*)p.y.p + b * p.y.b + (tt + i * kPass) * p.y.t + y_off;
                        if constexpr (S::kPiece == 16) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
                        else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
                    }
                }
            };
            if (whole_channels && tt + kTile <= t1) put_rows(std::true_type());
            else put_rows(std::false_type());
        }
        __syncwarp();
    }
#pragma unroll
    for (int q = 0; q < CH; ++q) {
        if (!on[q]) continue;
        auto put = [&](float* to, const float* v) {
#pragma unroll
            for (int i = 0; i < NS; i += 4)
                *reinterpret_cast<float4*>(to + j * NS + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        };
        if (kY) {
            if (p.h_out && t1 == p.T) put(p.h_out + (b * p.D + c[q]) * N, h[q]);
        } else {
            const long long at = (b * p.chunks + chunk) * p.D + c[q];
            put(p.chunk_h + at * N, h[q]);
            if constexpr (kBack) {
                bool finite = true;  // an infinite P leaves no finite sum
#pragma unroll
                for (int i = 0; i < NS; ++i) finite = finite && fabsf(back[q][i]) < INFINITY;
                if (!finite) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) back[q][i] = passed_back<T>(p, b, t0, t1, c[q], g, j * NS + i);
                }
            }
            if constexpr (kBack) put(p.chunk_g + at * N, back[q]);
            if (j == 0) p.chunk_s[at] = cut ? INFINITY : sum[q];
        }
    }
}

// ---- host ----------------------------------------------------------------------------

// A walk's lanes a channel and channels a lane.
struct Split {
    int lanes, channels;
    int cta() const { return kWarps * channels * 32 / lanes; }  // channels of a CTA
};

template <typename T, Mode MODE>
cudaError_t launch_scan(const SsmParams& p, Split split, unsigned grid, cudaStream_t s);

// The gradients' second walk (csrc/ssm_bwd.cuh).
template <typename T>
cudaError_t launch_gradients(const SsmBwdParams& p, unsigned grid, cudaStream_t s);

template <typename S>
cudaError_t launch_shape(const SsmParams& p, unsigned grid, cudaStream_t s) {
    if (S::kShared > 48 * 1024) {  // what a kernel may have without asking
        const cudaError_t e = cudaFuncSetAttribute(ssm_scan_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)S::kShared);
        if (e != cudaSuccess) return e;
    }
    TraceScope trace(S::MODE == kForward ? "ssm_kernel" : S::MODE == kState ? "ssm_state_kernel" : "ssm_summary_kernel",
                     s);
    ssm_scan_kernel<S><<<grid, kWarps * 32, S::kShared, s>>>(p);
    return cudaGetLastError();
}

template <typename T, Mode MODE>
cudaError_t launch_scan_here(const SsmParams& p, Split split, unsigned grid, cudaStream_t s) {
    const int ns = p.N / split.lanes;
#define LA_SSM_SHAPE(CH, NS, L) \
    if (split.channels == CH && ns == NS && split.lanes == L) return launch_shape<Shape<T, CH, NS, L, MODE>>(p, grid, s);
    LA_SSM_SHAPE(1, 8, 1)
    LA_SSM_SHAPE(2, 8, 2)
    LA_SSM_SHAPE(2, 8, 4)
    LA_SSM_SHAPE(2, 8, 8)
    if constexpr (MODE != kSummary) {
        LA_SSM_SHAPE(1, 4, 2)
        LA_SSM_SHAPE(1, 4, 4)
        LA_SSM_SHAPE(1, 4, 8)
    }
#undef LA_SSM_SHAPE
    return cudaErrorInvalidValue;
}

}  // namespace ssm
}  // namespace la
