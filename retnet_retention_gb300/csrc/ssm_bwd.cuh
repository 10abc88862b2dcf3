// The gradients of the selective scan, chunk by chunk.  With du = dy gate sigmoid(gate),
// u = c_t . h_t + skip x and e_t = exp(delta_t A), walking backward from the gradient of
// the state that leaves the chunk:
//
//   g_t = c_t du_t + e_(t+1) g_(t+1)
//   s = sum_n g b,  q = (e_t g_t) h_(t-1),  r = sum_n q A
//   dx = delta s + skip du,  ddt = (x s + r) softplus'(dt + dt_bias),  dgate = dy u silu'(gate)
//   dA = sum_t q delta,  db_n = sum over channels g delta x,  dc_n = sum over channels du h_t
//
// The walk over a chunk's blocks of kBlock tokens goes backward; a block's states are
// computed again from the state before it (the local one the summary walk left, plus what
// the chunk's entering state has become), and those of half a block kept in registers while it
// is walked backward: the first half's are computed twice, which costs less than the warps
// that the registers of a whole block would.
//
// 4 x 4096 tokens of 2048 channels of 16 states: 646 us of this walk, after 234 of the summary walk and
// 23 of the join, before 33 of the sums; bound by issue slots, 233 instructions for a token of a warp's 16
// channels, 58 of them packed, at 3 warps a scheduler (what 168 registers leave); HBM is at 16 %.
//
// A lane holds four states of two channels.  Sums over n cross L = N / 4 lanes, sums over
// channels (for db, dc) the other 32 / L: both give away half of what they hold at each
// step.  Which state a register holds is turned with the lane (n = 4 j + (i ^ turn)), and
// which channel, so that the halves to keep and to give have fixed registers.
#pragma once

#include "ssm.cuh"

namespace la {
namespace ssm {

constexpr int kBwdWarps = 4;

template <typename T_, int N_>
struct BwdShape {
    using T = T_;
    static constexpr int N = N_, L = N / 4, CL = 32 / L, WC = 2 * CL;  // lanes of a channel, pairs and channels of a warp
    static constexpr int kTurns = CL < 4 ? CL : 4;                     // ways the four states are turned
    static constexpr int M = L / 2, K = kBlock / M;                    // own tokens: every M-th, K of a block
    static constexpr int kRows = kBlock * WC, kShared = kBlock * 2 * N;  // entries of a tensor's block; of b and c
    static constexpr int kPiece = WC * (int)sizeof(T) < 16 ? WC * (int)sizeof(T) : 16, kElems = kPiece / (int)sizeof(T);
    static constexpr int kThreads = kBwdWarps * 32;
    // Channels lie in a warp's shared memory with the even ones first (place), so that lanes side by
    // side read side by side.
    __device__ static int place(int c) { return (c & 1) * CL + c / 2; }
    static constexpr int kStates = N + 4;  // floats from a channel's states to the next's: 8 lanes meet no bank twice
    // A warp's shared memory, in bytes.  Twice: the rows of x, dt, gate and dy of its channels, the
    // local states before the block and their sums of delta.  Once, for each token and channel: delta and
    // delta x; du; x; the slopes of dt and gate.
    static constexpr int kStageT = 4 * kRows * (int)sizeof(T);
    static constexpr int kStage = kStageT + WC * kStates * 4 + (WC * 4 + 15) / 16 * 16;
    static constexpr int kWarp = 2 * kStage + kRows * (8 + 4 + 4 + 8);
    // The CTA's.  Twice: the rows of b and c, and these as fp32, a copy for each turn (64 bytes apart
    // modulo 128, so that two copies meet no bank twice).  Each warp's sums over its channels, for one
    // block and the next (N = 64: one).
    static constexpr int kCopy = kShared + 16;  // floats
    static constexpr int kWide = kTurns * kCopy;
    static constexpr int kColumnSets = N == 64 ? 1 : 2;
    static constexpr int kBytes = kBwdWarps * kWarp + 2 * (kShared * (int)sizeof(T) + kWide * 4) +
                                  kColumnSets * kBwdWarps * kShared * 4;
};

template <typename S>
__global__ void __launch_bounds__(kBwdWarps * 32, 3) ssm_gradients_kernel(const __grid_constant__ SsmBwdParams bp) {
    using T = typename S::T;
    constexpr int N = S::N, CL = S::CL, WC = S::WC, U = kBlock, M = S::M, K = S::K, kThreads = S::kThreads;
    const SsmParams& p = bp.f;
    tc::griddep_launch_dependents();
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = lane / CL, cl = lane % CL;
    unsigned char* const mine = smem + w * S::kWarp;
    float2* const steps = reinterpret_cast<float2*>(mine + 2 * S::kStage);  // delta, delta x
    float2* const slopes = steps + S::kRows;
    float* const dus = reinterpret_cast<float*>(slopes + S::kRows);
    float* const xs = dus + S::kRows;
    T* const raw = reinterpret_cast<T*>(smem + kBwdWarps * S::kWarp);       // [2][token][2 N]
    float* const wides = reinterpret_cast<float*>(raw + 2 * S::kShared);    // [2][turn][token][2 N]
    float* const columns = wides + 2 * S::kWide;                            // [set][warp][token][2 N]
    unsigned unit = blockIdx.x;
    const unsigned tile = unit % (unsigned)(p.tiles * p.G);
    unit /= (unsigned)(p.tiles * p.G);
    const int chunk = (int)(unit % (unsigned)p.chunks);
    const long long b = unit / (unsigned)p.chunks;
    const int g_at = (int)(tile / (unsigned)p.tiles);
    const int first = (int)(tile % (unsigned)p.tiles) * (kBwdWarps * WC) + w * WC;
    const int turn = cl & (S::kTurns - 1);
    // register q of two: channel 2 cl + (q ^ (j & 1)), so that register 0 is the lane's own
    const int mine_c = 2 * cl + (j & 1), other_c = 2 * cl + (1 ^ (j & 1));
    const int mine_at = S::place(mine_c), other_at = S::place(other_c);
    const bool on = first + mine_c < p.channels;  // D / G is even: both or neither
    const int c0 = g_at * p.channels + first;  // the warp's first channel
    const int t0 = chunk * p.chunk, t1 = (int)min((long long)t0 + p.chunk, (long long)p.T);
    float2 A[2][2], g[2][2], hin[2][2], dA[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int c = on ? c0 + (q == 0 ? mine_c : other_c) : 0;
        const long long at = ((b * p.chunks + chunk) * p.D + c) * N;
        // four neighbouring states, turned
        auto states = [&](const float* from, float2 (&to)[2]) {
            float4 f = on ? *reinterpret_cast<const float4*>(from + 4 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (turn & 1) f = make_float4(f.y, f.x, f.w, f.z);
            if (turn & 2) f = make_float4(f.z, f.w, f.x, f.y);
            to[0] = make_float2(f.x, f.y);
            to[1] = make_float2(f.z, f.w);
        };
        states(p.A + (size_t)c * N, A[q]);
        states(p.chunk_h + at, hin[q]);
        states(p.chunk_g + at, g[q]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            A[q][i] = __fmul2_rn(A[q][i], both(kLog2e));
            dA[q][i] = make_float2(0.f, 0.f);
        }
    }
    const int own_c = on ? c0 + mine_c : 0, own = j >> 1;  // own tokens of a block: k M + own
    const float skip = p.skip ? p.skip[own_c] : 0.f, bias = p.bias ? p.bias[own_c] : 0.f;
    float dskip = 0.f, dbias = 0.f;
    const bool gated = p.gate.p != nullptr;

    int position = 1;
    auto copy_block = [&](int buf, int t) {  // t below t0: nothing
        unsigned char* const stage = mine + buf * S::kStage;
        if (t >= t0) {
            constexpr int kPerRow = WC / S::kElems, kPieces = U * kPerRow;
#pragma unroll
            for (int i = 0; i < (4 * kPieces + 31) / 32; ++i) {
                const int q = i * 32 + lane, k = q / kPieces, row = q % kPieces / kPerRow, at = q % kPerRow * S::kElems;
                if ((4 * kPieces) % 32 == 0 || q < 4 * kPieces) {
                    const SsmRows& r = k == 0 ? p.x : k == 1 ? p.dt : k == 2 ? (gated ? p.gate : p.x) : p.dy;
                    const bool valid = t + row < t1 && first + at < p.channels;
                    copy_piece<S::kPiece>((T*)stage + k * S::kRows + row * WC + at,
                                          (const T*)r.p + b * r.b + (valid ? t + row : 0) * r.t +
                                              (valid ? g_at * p.channels + first + at : 0), valid);
                }
            }
            // eight entries of b or c a thread, which brings them to fp32 itself
#pragma unroll
            for (int i = 0; i < (S::kShared / 8 + kThreads - 1) / kThreads; ++i) {
                const int q = i * kThreads + threadIdx.x, row = q / (2 * N / 8), part = q % (2 * N / 8);
                if ((S::kShared / 8) % kThreads == 0 || q < S::kShared / 8) {
                    const SsmRows& r = part < N / 8 ? p.bm : p.cm;
                    const bool valid = t + row < t1;
                    const T* const from =
                        (const T*)r.p + b * r.b + (valid ? t + row : 0) * r.t + g_at * N + part % (N / 8) * 8;
#pragma unroll
                    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
                        copy16(raw + buf * S::kShared + q * 8 + k * 4, from + k * 4, valid);
                }
            }
            if (t > t0) {
                const long long at = (b * p.blocks + t / U) * p.D + c0;
                float* const states = reinterpret_cast<float*>(stage + S::kStageT);
#pragma unroll
                for (int i = 0; i < (WC * N / 4 + 31) / 32; ++i) {
                    const int q = i * 32 + lane, c = q * 4 / N;
                    if ((WC * N / 4) % 32 == 0 || q < WC * N / 4) {
                        const bool valid = first + c < p.channels;
                        copy16(states + S::place(c) * S::kStates + q * 4 % N, valid ? p.block_h + at * N + q * 4 : p.block_h,
                               valid);
                    }
                }
                if (lane < WC / 4) {
                    const bool valid = first + lane * 4 < p.channels;
                    copy16(states + WC * S::kStates + lane * 4, valid ? p.block_s + at + lane * 4 : p.block_s, valid);
                }
            }
            if (p.positions) position = lane < U && t + lane < t1 ? p.positions[b * p.T + t + lane] : 1;
        }
        copies_commit();
    };
    // dx, ddt and dgate of the block at t, which lie where x, dt and gate were
    auto put_block = [&](int buf, int t) {
        const unsigned char* const stage = mine + buf * S::kStage;
        constexpr int kPerRow = WC / S::kElems, kPieces = U * kPerRow;
#pragma unroll
        for (int i = 0; i < (3 * kPieces + 31) / 32; ++i) {
            const int q = i * 32 + lane, k = q / kPieces, row = q % kPieces / kPerRow, at = q % kPerRow * S::kElems;
            if (q < (gated ? 3 : 2) * kPieces && t + row < t1 && first + at < p.channels) {
                const SsmRows& r = k == 0 ? bp.dx : k == 1 ? bp.ddt : bp.dgate;
                const T* const from = (const T*)stage + k * S::kRows + row * WC + at;
                T* const to = (T*)r.p + b * r.b + (t + row) * r.t + c0 + at;
                if constexpr (S::kPiece == 16) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
                else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
            }
        }
    };
    // the warps' sums over channels of the block at t
    auto add_up = [&](int t, int from) {
        const float* const set = columns + from % S::kColumnSets * (kBwdWarps * S::kShared);
        for (int i = threadIdx.x; i < S::kShared; i += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kBwdWarps; ++k) v += set[k * S::kShared + i];
            const int tok = i / (2 * N), col = i % (2 * N);
            if (t + tok < t1) bp.part_bc[(((long long)tile * p.B + b) * p.T + t + tok) * (2 * N) + col] = v;
        }
    };
    const int last = t0 + (t1 - t0 - 1) / U * U;
    copy_block(0, last);
    int buf = 0;
    for (int t = last; t >= t0; t -= U, buf ^= 1) {
        const unsigned starts = p.positions ? __ballot_sync(0xffffffffu, position == 0) : 0;
        copy_block(buf ^ 1, t - U);
        copies_wait<1>();
        __syncwarp();
        unsigned char* const stage = mine + buf * S::kStage;
        // the block's own elementwise values
        constexpr int kPairs = (K + 1) / 2;  // two own tokens at a time (one, where it is the only one)
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            const int row = (2 * k * M + own) * WC, row2 = K == 1 ? row : row + M * WC;
            const T* const from = (const T*)stage + mine_c;
            auto pair = [&](int tensor) {
                return make_float2(load_elem(from + tensor * S::kRows, row), load_elem(from + tensor * S::kRows, row2));
            };
            const float2 x = pair(0), v = __fadd2_rn(pair(1), both(bias));
            float2 d = v, du = pair(3), slope = both(1.f), gate_slope = both(0.f);
            if (p.softplus) d = softplus2<T>(v, &slope);
            // no token: the state stays as it is (x, dy and so on are zeros)
            if (t + 2 * k * M + own >= t1) d.x = 0.f;
            if (t + (2 * k + 1) * M + own >= t1) d.y = 0.f;
            if (gated) {
                const float2 z = pair(2), s = sigmoid2<T>(z), a = __fmul2_rn(z, s);
                gate_slope = __fmul2_rn(du, __ffma2_rn(a, __ffma2_rn(s, both(-1.f), both(1.f)), s));
                du = __fmul2_rn(du, a);
            }
            const float2 dx = __fmul2_rn(d, x);
            steps[row + mine_at] = make_float2(d.x, dx.x);
            slopes[row + mine_at] = make_float2(slope.x, gate_slope.x);
            dus[row + mine_at] = du.x;
            xs[row + mine_at] = x.x;
            if (K > 1) {
                steps[row2 + mine_at] = make_float2(d.y, dx.y);
                slopes[row2 + mine_at] = make_float2(slope.y, gate_slope.y);
                dus[row2 + mine_at] = du.y;
                xs[row2 + mine_at] = x.y;
            }
        }
        // b and c to fp32, a copy for each turn: entry i of a group of four is entry i ^ turn
        float* const wide = wides + buf * S::kWide;
#pragma unroll
        for (int i = 0; i < (S::kShared / 8 + kThreads - 1) / kThreads; ++i) {
            const int q = i * kThreads + threadIdx.x;
            if ((S::kShared / 8) % kThreads == 0 || q < S::kShared / 8) {
                float2 v[4];
                floats8<false>(raw8<true>(raw + buf * S::kShared + q * 8, 0, 4), v);
#pragma unroll
                for (int k = 0; k < S::kTurns; ++k) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float f[4] = {v[2 * half].x, v[2 * half].y, v[2 * half + 1].x, v[2 * half + 1].y};
                        *reinterpret_cast<float4*>(wide + k * S::kCopy + q * 8 + 4 * half) =
                            make_float4(f[0 ^ k], f[1 ^ k], f[2 ^ k], f[3 ^ k]);
                    }
                }
            }
        }
        // the state before the block: the local one and the chunk's entering one, decayed
        float2 enter[2][2];
        {
            const float* const states = reinterpret_cast<const float*>(stage + S::kStageT);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float sum = t > t0 ? states[WC * S::kStates + (q == 0 ? mine_c : other_c)] : 0.f;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (t > t0) f = *reinterpret_cast<const float4*>(states + (q == 0 ? mine_at : other_at) * S::kStates + 4 * j);
                if (turn & 1) f = make_float4(f.y, f.x, f.w, f.z);
                if (turn & 2) f = make_float4(f.z, f.w, f.x, f.y);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 local = i == 0 ? make_float2(f.x, f.y) : make_float2(f.z, f.w);
                    const float2 e = half_decay2(sum, A[q][i]);
                    enter[q][i] = sum == INFINITY ? local : __ffma2_rn(e, __fmul2_rn(e, hin[q][i]), local);
                }
            }
        }
        __syncthreads();
        if (t != last) {
            add_up(t + U, buf ^ 1);  // of the block before this one
            if (S::kColumnSets == 1) __syncthreads();
        }
        const float* const bc = wide + turn * S::kCopy + 4 * j;
        auto walk = [&](auto careful) {
            constexpr bool kCareful = decltype(careful)::value;
            constexpr int H = U / 2;  // the states of half a block are kept at a time
            auto forward = [&](int u, const float2 (&from)[2][2], float2 (&to)[2][2]) {
                const float4 bv = *reinterpret_cast<const float4*>(bc + u * 2 * N);
                const float2 b2[2] = {make_float2(bv.x, bv.y), make_float2(bv.z, bv.w)};
                const bool start = kCareful && (starts >> u & 1);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float2 v = steps[u * WC + (q == 0 ? mine_at : other_at)];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = __ffma2_rn(both(v.x), A[q][i], both(kRaise)), add = __fmul2_rn(both(v.y), b2[i]);
                        to[q][i] = __ffma2_rn(make_float2(exp2_fast(x.x), exp2_fast(x.y)), from[q][i], add);
                        if (start) to[q][i] = add;
                    }
                }
            };
            float2 hs[H + 1][2][2];
            auto keep = [&](const float2 (&v)[2][2]) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i) hs[0][q][i] = v[q][i];
            };
            keep(enter);
#pragma unroll
            for (int u = 0; u < H; ++u) {
                float2 h[2][2];
                forward(u, hs[0], h);
                keep(h);
            }
#pragma unroll 1
            for (int u0 = H; u0 >= 0; u0 -= H) {
                if (u0 == 0) keep(enter);
#pragma unroll
                for (int u = 0; u < H; ++u) forward(u0 + u, hs[u], hs[u + 1]);
                float sv[H], rv[H], yv[H];
#pragma unroll
                for (int u = H - 1; u >= 0; --u) {
                    const float4 bv = *reinterpret_cast<const float4*>(bc + (u0 + u) * 2 * N);
                    const float4 cv = *reinterpret_cast<const float4*>(bc + (u0 + u) * 2 * N + N);
                    const float2 b2[2] = {make_float2(bv.x, bv.y), make_float2(bv.z, bv.w)};
                    const float2 c2[2] = {make_float2(cv.x, cv.y), make_float2(cv.z, cv.w)};
                    const bool start = kCareful && (starts >> (u0 + u) & 1);
                    float2 s[2], r[2], y[2], db2[2], dc2[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int at = (u0 + u) * WC + (q == 0 ? mine_at : other_at);
                        const float2 val = steps[at];
                        const float du = dus[at];
                        const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 h = hs[u + 1][q][i];
                            g[q][i] = __ffma2_rn(c2[i], both(du), g[q][i]);
                            s[q] = i == 0 ? __fmul2_rn(g[q][i], b2[i]) : __ffma2_rn(g[q][i], b2[i], s[q]);
                            y[q] = i == 0 ? __fmul2_rn(h, c2[i]) : __ffma2_rn(h, c2[i], y[q]);
                            db2[i] = q == 0 ? __fmul2_rn(g[q][i], both(val.y)) : __ffma2_rn(g[q][i], both(val.y), db2[i]);
                            dc2[i] = q == 0 ? __fmul2_rn(h, both(du)) : __ffma2_rn(h, both(du), dc2[i]);
                            const float2 x = __ffma2_rn(both(val.x), A[q][i], both(kRaise));
                            g[q][i] = __fmul2_rn(g[q][i], make_float2(exp2_fast(x.x), exp2_fast(x.y)));
                            if (start) g[q][i] = zero;
                            float2 qq = __fmul2_rn(g[q][i], hs[u][q][i]);
                            if (start) qq = zero;
                            r[q] = i == 0 ? __fmul2_rn(qq, A[q][i]) : __ffma2_rn(qq, A[q][i], r[q]);
                            dA[q][i] = __ffma2_rn(qq, both(val.x), dA[q][i]);
                        }
                    }
                    // over n: the own channel's register is kept
                    sv[u] = s[0].x + s[0].y + __shfl_xor_sync(0xffffffffu, s[1].x + s[1].y, CL);
                    rv[u] = r[0].x + r[0].y + __shfl_xor_sync(0xffffffffu, r[1].x + r[1].y, CL);
                    yv[u] = y[0].x + y[0].y + __shfl_xor_sync(0xffffffffu, y[1].x + y[1].y, CL);
                    // over channels
                    float db[4] = {db2[0].x, db2[0].y, db2[1].x, db2[1].y}, dc[4] = {dc2[0].x, dc2[0].y, dc2[1].x, dc2[1].y};
                    if (CL >= 4) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            db[i] += __shfl_xor_sync(0xffffffffu, db[i + 2], 2);
                            dc[i] += __shfl_xor_sync(0xffffffffu, dc[i + 2], 2);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < (CL >= 4 ? 1 : 3); i += 2) {
                        db[i] += __shfl_xor_sync(0xffffffffu, db[i + 1], 1);
                        dc[i] += __shfl_xor_sync(0xffffffffu, dc[i + 1], 1);
                    }
                    float* const to = columns + ((buf % S::kColumnSets * kBwdWarps + w) * U + u0 + u) * 2 * N + 4 * j;
                    if (CL > 4) {
                        // half of the lanes keep db, half dc
                        const bool c_half = cl & 4;
                        float v = (c_half ? dc[0] : db[0]) + __shfl_xor_sync(0xffffffffu, c_half ? db[0] : dc[0], 4);
#pragma unroll
                        for (int gap = 8; gap < CL; gap *= 2) v += __shfl_xor_sync(0xffffffffu, v, gap);
                        if (CL == 8 || cl < 8) to[(c_half ? N : 0) + turn] = v;
                    } else if (CL == 4) {
                        to[turn] = db[0];
                        to[N + turn] = dc[0];
                    } else {
                        to[turn] = db[0];
                        to[2 + turn] = db[2];
                        to[N + turn] = dc[0];
                        to[N + 2 + turn] = dc[2];
                    }
                }
                // the own tokens of these: their sums over n come to this lane
                constexpr int kOwn = M <= H ? H / M : 1;
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    float s, r, y;
                    int at_u;
                    bool mine_now = on;
                    if constexpr (M <= H) {
                        float sk[M], rk[M], yk[M];
#pragma unroll
                        for (int i = 0; i < M; ++i) sk[i] = sv[k * M + i], rk[i] = rv[k * M + i], yk[i] = yv[k * M + i];
                        s = share_sums<M>(sk, own, 2 * CL), r = share_sums<M>(rk, own, 2 * CL);
                        y = share_sums<M>(yk, own, 2 * CL);
                        at_u = u0 + k * M + own;
                    } else {  // M = 8: the lanes of the other half hold the same tokens' other sums
                        s = share_sums<H>(sv, own & (H - 1), 2 * CL), r = share_sums<H>(rv, own & (H - 1), 2 * CL);
                        y = share_sums<H>(yv, own & (H - 1), 2 * CL);
                        s += __shfl_xor_sync(0xffffffffu, s, H * 2 * CL);
                        r += __shfl_xor_sync(0xffffffffu, r, H * 2 * CL);
                        y += __shfl_xor_sync(0xffffffffu, y, H * 2 * CL);
                        at_u = u0 + (own & (H - 1));
                        mine_now = on && (own >= H) == (u0 > 0);
                    }
                    if (mine_now && t + at_u < t1) {  // what is not there adds nothing to the sums
                        constexpr float kLn2 = 0.69314718055994531f;  // A holds log2 e
                        const int at = at_u * WC + mine_at;
                        const float2 step = steps[at], slope = slopes[at];
                        const float x = xs[at], du = dus[at];
                        const float ddt = fmaf(x, s, r * kLn2) * slope.x;
                        T* const to = (T*)stage + at_u * WC + mine_c;
                        store_elem(to, 0, fmaf(step.x, s, skip * du));
                        store_elem(to, S::kRows, ddt);
                        if (gated) store_elem(to, 2 * S::kRows, slope.y * fmaf(skip, x, y));
                        dskip = fmaf(du, x, dskip);
                        dbias += ddt;
                    }
                }
            }
        };
        if (starts == 0) walk(std::false_type());
        else walk(std::true_type());
        __syncwarp();
        put_block(buf, t);
        __syncwarp();
    }
    __syncthreads();
    add_up(t0, buf ^ 1);
    const long long part = b * p.chunks + chunk;
    if (on) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int c = c0 + (q == 0 ? mine_c : other_c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = 4 * j + (i ^ turn);
                const float2 a = dA[q][i / 2], gg = g[q][i / 2];
                if (bp.part_A) bp.part_A[(part * p.D + c) * N + n] = i % 2 ? a.y : a.x;
                if (bp.dh0 && chunk == 0) bp.dh0[(b * p.D + c) * N + n] = i % 2 ? gg.y : gg.x;
            }
        }
    }
#pragma unroll
    for (int gap = 1; gap < M; gap *= 2) {
        dskip += __shfl_xor_sync(0xffffffffu, dskip, gap * 2 * CL);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, gap * 2 * CL);
    }
    if (on && own == 0) {
        if (bp.part_skip) bp.part_skip[part * p.D + own_c] = dskip;
        if (bp.part_bias) bp.part_bias[part * p.D + own_c] = dbias;
    }
}

template <typename S>
cudaError_t launch_gradients_shape(const SsmBwdParams& p, unsigned grid, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(ssm_gradients_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               S::kBytes);
    if (e != cudaSuccess) return e;
    TraceScope trace("ssm_gradients_kernel", s);
    ssm_gradients_kernel<S><<<grid, kBwdWarps * 32, S::kBytes, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gradients_here(const SsmBwdParams& p, unsigned grid, cudaStream_t s) {
    switch (p.f.N) {
        case 8: return launch_gradients_shape<BwdShape<T, 8>>(p, grid, s);
        case 16: return launch_gradients_shape<BwdShape<T, 16>>(p, grid, s);
        case 32: return launch_gradients_shape<BwdShape<T, 32>>(p, grid, s);
        default: return launch_gradients_shape<BwdShape<T, 64>>(p, grid, s);
    }
}

}  // namespace ssm
}  // namespace la
