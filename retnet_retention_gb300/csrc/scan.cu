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
// memory), and every thread then replays its rows from the state that enters them.
// x and log_a are read once and h written once; no workspace, no atomics, no waits on
// global memory, and the order of all sums is fixed by the launch shape.
//
// A decay of exactly zero (log_a = -inf) restarts its channel: the old state is
// dropped by a selection, not multiplied by zero, so that an infinity or a NaN in
// it, or in a decay before, does not pass.  Nothing else drops one: a run's product
// that underflows without a zero among its decays is held at the least fp32 number (an
// error of 2^-149 of the state), so that what an infinity or a NaN reaches does not
// depend on the runs' lengths.
//
// Bound by HBM: log_a 4, x 2, h 2 bytes an entry (bf16).  State, products and sums
// are fp32; h is rounded where it is stored, never the state that is carried on.
//
// A warp copies its own rows two rounds ahead (asynchronous copies into shared memory,
// no barrier beyond the warp); with plain loads at the head of a round 8 x 8192 x 4096
// took 639 us, with the ring 353, with addresses that run along instead of being
// recomputed 327.  The CTAs of a cluster exchange by remote stores that count on the
// receiver's barrier: a cluster barrier waits for the round's stores of h as well (1 x
// 65536 x 1024: 189 us against 168).  Sending a round's runs before the round ahead of
// it is finished gained nothing (142 against 141 us on one GPU): the exchange is not what
// a round waits for.
//
// One GB300, bf16: 8 x 8192 x 4096 326 us (6.6 TB/s, 0.97 of a copy's rate; 333 on another
// card), 1 x 65536 x 1024 109 us (4.9 TB/s: 32 tiles of channels in clusters of 8 fill 256
// of 304 places, 1.19 of the 1.37 it lies above its floor; the rest is a round's chain of
// copies, exponentials, barrier, exchange and replay with 12 warps an SM, issue slots half
// used), gradients of 4 x 4096 x 2048 73 us (6.4 TB/s).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

using namespace tc;

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
    int* dev_status;     // or null
    uint64_t limit_ns;   // of a wait for the cluster's runs
    bool mute;           // test switch: push nothing, so that the waits run out
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
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// Write v to the same shared address in CTA `rank` of the cluster and count its bytes
// on that CTA's barrier: unlike a cluster barrier this waits for nothing else, in
// particular not for the round's stores of h.
__device__ __forceinline__ void push(const float2* at, const uint64_t* bar, unsigned rank, float2 v) {
    asm volatile(
        "{\n\t.reg .b32 ra, rb;\n\tmapa.shared::cluster.u32 ra, %0, %2;\n\t"
        "mapa.shared::cluster.u32 rb, %1, %2;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [ra], {%3, %4}, [rb];\n\t}" ::"r"(
            smem_addr(at)),
        "r"(smem_addr(bar)), "r"(rank), "f"(v.x), "f"(v.y)
        : "memory");
}
__device__ __forceinline__ bool arrived(const uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
// Wait for the cluster's runs of a round.  The CTAs of a cluster run at the same time,
// so this ends within microseconds; after the limit it gives up, and so do the
// CTA's other warps and later rounds, which then run on without the runs.
__device__ __noinline__ void wait_long(const uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                       volatile int* gave_up) {
    const uint64_t t0 = global_timer_ns();
    while (!arrived(bar, parity)) {
        if (*gave_up) return;
        if (global_timer_ns() - t0 > limit_ns) {
            *gave_up = 1;
            return;
        }
    }
}
__device__ __forceinline__ void wait_runs(const uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                          volatile int* gave_up) {
    if (!arrived(bar, parity)) wait_long(bar, parity, limit_ns, gave_up);
}

// The state s after a run (A, b).
__device__ __forceinline__ float after(float A, float b, float s) {
    return A == 0.f ? b : fmaf(A, s, b);
}

constexpr float kLeast = 1.401298464e-45f;  // 2^-149, the least fp32 number

// V neighbouring entries of a row in shared memory, as fp32.
template <int V>
__device__ __forceinline__ void row_floats(const float* p, float (&v)[V]) {
    if (V == 2) {
        const float2 r = *reinterpret_cast<const float2*>(p);
        v[0] = r.x;
        v[V - 1] = r.y;
    } else {
        v[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void row_floats(const __nv_bfloat16* p, float (&v)[V]) {
    if (V == 2) {
        const uint32_t r = *reinterpret_cast<const uint32_t*>(p);
        v[0] = __uint_as_float(r << 16);
        v[V - 1] = __uint_as_float(r & 0xffff0000u);
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
    if (V == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[V - 1]);
    else *p = v[0];
}
template <int V>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&v)[V]) {
    if (V == 2) *reinterpret_cast<uint32_t*>(p) = bf16x2_bits(v[0], v[V - 1]);
    else *p = __float2bfloat16_rn(v[0]);
}

// One kernel's shape: V channels a lane (a tile has C = 32 V), R rows a thread and
// round, W warps, S rounds of rows in the ring, CTAS on an SM.
template <typename T, int V_, int R_, int W_, int S_, int CTAS_, bool BWD_>
struct Shape {
    using Elem = T;
    static constexpr int V = V_, R = R_, W = W_, S = S_, kCtas = CTAS_, C = 32 * V_;
    static constexpr bool BWD = BWD_;
    static constexpr int kRun = W * R;  // rows a CTA takes a round
    static constexpr size_t kLog = (size_t)kRun * C * sizeof(float);
    static constexpr size_t kX = (size_t)kRun * C * sizeof(T);
    static constexpr size_t kStage = kLog + kX * (BWD ? 2 : 1);
    static constexpr size_t kRuns = 2 * (size_t)(W + kMaxCluster) * C * sizeof(float2);
    static constexpr size_t kShared = S * kStage + kRuns;
};

// One cluster walks one tile of channels of one sequence; backward, it walks from the
// last token to the first.  A warp copies the rows it works on itself, a ring of S
// rounds ahead, so that the ring needs no barrier beyond the warp's own.
template <typename K>
__global__ void __launch_bounds__(K::W * 32, K::kCtas) scan_kernel(const __grid_constant__ ScanParams p) {
    using T = typename K::Elem;
    constexpr int V = K::V, R = K::R, W = K::W, S = K::S, C = K::C;
    constexpr bool BWD = K::BWD;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[2];  // the cluster's runs of even and odd rounds
    __shared__ int gave_up;
    float2* warp_run = reinterpret_cast<float2*>(smem + S * K::kStage);  // [2][W][C]
    float2* cta_run = warp_run + 2 * W * C;                              // [2][kMaxCluster][C]
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const unsigned rank = cluster_rank(), n = cluster_size();
    const unsigned unit = blockIdx.x / n;  // not %clusterid: past 2^24 it came back rounded to 24 bits
    const unsigned b = unit / (unsigned)p.tiles, tile = unit - b * (unsigned)p.tiles;
    const int first = (int)tile * C, c0 = first + lane * V;
    const bool on = c0 < p.D;
    // Rows are counted in walking order: row u is token u, or T - 1 - u backward.
    const long long step = BWD ? -(long long)p.D : (long long)p.D, seq = (long long)b * p.T * p.D;
    const long long origin = seq + (BWD ? (p.T - 1ll) * p.D : 0);  // row 0
    const long long mine = (long long)rank * K::kRun + w * R, leap = (long long)n * K::kRun;

    // A warp copies 16-byte pieces: of log_a (kLogRows rows at a time), of x (dh), and
    // backward of h one token earlier.  A lane's piece keeps its column.
    constexpr int kLogRows = 32 / (C / 4), kElems = 16 / (int)sizeof(T), kRows = 32 / (C / kElems);
    static_assert(R % kLogRows == 0 && R % kRows == 0, "whole passes");
    const int log_row = lane / (C / 4), log_c = first + lane % (C / 4) * 4;
    const int x_row = lane / (C / kElems), x_c = first + lane % (C / kElems) * kElems;
    const bool log_on = log_c < p.D, x_on = x_c < p.D;
    const float* log_src = p.log_a + origin + (mine + log_row) * step + (log_on ? log_c : 0);
    const T* x_src = (const T*)p.x + origin + (mine + x_row) * step + (x_on ? x_c : 0);
    const T* h_src = (const T*)p.h_in + origin + (mine + x_row + 1) * step + (x_on ? x_c : 0);
    long long u_src = mine;  // the warp's first row of the next round to copy
    unsigned char* const slot = smem + (size_t)w * R * C * sizeof(float) + lane * 16;
    unsigned char* const x_slot = smem + K::kLog + (size_t)w * R * C * sizeof(T) + lane * 16;
    // Copy the next round's rows into stage s.  Rows past the end arrive as zeros:
    // log_a 0, x 0 leave the state as it is.
    auto fetch = [&](int s) {
        unsigned char* const to = slot + s * K::kStage;
        unsigned char* const x_to = x_slot + s * K::kStage;
        auto pieces = [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;  // all rows inside, the last token not among them
#pragma unroll
            for (int i = 0; i < R / kLogRows; ++i) {
                const bool valid = log_on && (kWhole || u_src + i * kLogRows + log_row < p.T);
                copy16(to + i * 512, kWhole || valid ? log_src + i * kLogRows * step : p.log_a, valid);
            }
#pragma unroll
            for (int i = 0; i < R / kRows; ++i) {
                const long long u = u_src + i * kRows + x_row;
                const bool valid = x_on && (kWhole || u < p.T), before = x_on && (kWhole || u + 1 < p.T);
                copy16(x_to + i * 512, kWhole || valid ? x_src + i * kRows * step : (const T*)p.x, valid);
                if (BWD)
                    copy16(x_to + K::kX + i * 512,
                           kWhole || before ? h_src + i * kRows * step : (const T*)p.h_in, before);
            }
        };
        if (u_src + R < p.T) pieces(std::true_type());
        else pieces(std::false_type());
        u_src += leap;
        log_src += leap * step;
        x_src += leap * step;
        h_src += leap * step;
    };

    const uint32_t runs_bytes = n * C * sizeof(float2);
    if (n > 1 && threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[i], 1);
            mbar_arrive_expect_tx(&bars[i], runs_bytes);
        }
        fence_mbar_init();
    }
    const int rounds = (int)(((long long)p.T + (long long)K::kRun * n - 1) / ((long long)K::kRun * n));
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (s < rounds) fetch(s);
        copies_commit();
    }
    float state[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        state[j] = on && p.s0 ? p.s0[(size_t)b * p.D + c0 + j] : 0.f;
    if (n > 1) cluster_barrier();  // every CTA of the cluster runs, its barriers set up, before any is written to

    const float* const log_run = reinterpret_cast<const float*>(smem) + w * R * C + lane * V;
    const T* const x_run = reinterpret_cast<const T*>(smem + K::kLog) + w * R * C + lane * V;
    T* y = (T*)p.y + origin + mine * step + (on ? c0 : 0);
    float* dlog_a = BWD ? p.dlog_a + origin + mine * step + (on ? c0 : 0) : nullptr;
    long long u0 = mine;
    for (int round = 0, stage = 0; round < rounds; ++round, stage = stage + 1 == S ? 0 : stage + 1) {
        const int par = round & 1;  // the round's half of the exchange buffers
        float a[R][V], v[R][V], hp[BWD ? R : 1][V];
        copies_wait<S - 1>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            row_floats<V>(log_run + stage * (K::kStage / sizeof(float)) + i * C, a[i]);
            row_floats<V>(x_run + stage * (K::kStage / sizeof(T)) + i * C, v[i]);
            if (BWD)
                row_floats<V>(x_run + stage * (K::kStage / sizeof(T)) + K::kX / sizeof(T) + i * C,
                              hp[BWD ? i : 0]);
        }
        __syncwarp();
        if (round + S < rounds) fetch(stage);
        copies_commit();
        if (BWD && p.h0 && u0 < p.T && u0 + R >= p.T && on) {  // token 0 follows h0
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (u0 + i == p.T - 1)
#pragma unroll
                    for (int j = 0; j < V; ++j) hp[BWD ? i : 0][j] = p.h0[(size_t)b * p.D + c0 + j];
        }
        float A[V], bb[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.f, bb[j] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                a[i][j] = expf(a[i][j]);
                bb[j] = BWD && i == 0 ? v[i][j] : fmaf(a[BWD && i > 0 ? i - 1 : i][j], bb[j], v[i][j]);
                A[j] *= a[i][j];
            }
        // a zero among the decays makes the product zero, or a NaN where another one is
        // NaN or infinite: only then (or after an underflow) do the restarts' selections
        // run, for the whole warp
        bool zero = false;
#pragma unroll
        for (int j = 0; j < V; ++j) zero |= !(A[j] > 0.f);
        const bool cut = __any_sync(0xffffffffu, zero);
        if (cut) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float least = kLeast;
                bb[j] = 0.f;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    least = fminf(least, a[i][j]);
                    bb[j] = BWD && i == 0 ? v[i][j] : after(a[BWD && i > 0 ? i - 1 : i][j], v[i][j], bb[j]);
                }
                A[j] = fmaxf(A[j], least);  // a number: after a NaN decay and no restart bb is the NaN
            }
        }
        if (BWD) {  // so far the run's last dx: what it passes on
#pragma unroll
            for (int j = 0; j < V; ++j) bb[j] = a[R - 1][j] == 0.f ? 0.f : a[R - 1][j] * bb[j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            warp_run[(par * W + w) * C + lane * V + j] = make_float2(A[j], bb[j]);
        __syncthreads();
        // the run before this warp's in the CTA, and the whole CTA's
        float pA[V], pb[V], tA[V], tb[V], p_least[V], least[V];  // least: 0 once a run holds a restart
#pragma unroll
        for (int j = 0; j < V; ++j)
            tA[j] = pA[j] = 1.f, tb[j] = pb[j] = 0.f, least[j] = p_least[j] = kLeast;
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 r = warp_run[(par * W + i) * C + lane * V + j];
                if (i == w) pA[j] = tA[j], pb[j] = tb[j], p_least[j] = least[j];
                tb[j] = after(r.x, r.y, tb[j]);
                tA[j] *= r.x;
                least[j] = fminf(least[j], r.x);
            }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            tA[j] = fmaxf(tA[j], least[j]);
            pA[j] = fmaxf(pA[j], p_least[j]);
        }
        float s[V];
        if (n > 1) {
            // A slot and its barrier are used again two rounds later.  A CTA pushes its
            // run of round r + 2 only when it has all runs of round r + 1, and a CTA pushes
            // that one behind the __syncthreads that all its warps reach with round r read.
            for (unsigned to = p.mute ? n : w; to < n; to += W)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    push(&cta_run[(par * kMaxCluster + rank) * C + lane * V + j], &bars[par], to,
                         make_float2(tA[j], tb[j]));
            wait_runs(&bars[par], (round >> 1) & 1, p.limit_ns, &gave_up);
            float2 g[kMaxCluster][V];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (r < n) g[r][j] = cta_run[(par * kMaxCluster + r) * C + lane * V + j];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                if (r < n) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if (r == rank) s[j] = after(pA[j], pb[j], state[j]);
                        state[j] = after(g[r][j].x, g[r][j].y, state[j]);
                    }
                }
            }
            if (threadIdx.x == 0 && !*(volatile int*)&gave_up)
                mbar_arrive_expect_tx(&bars[par], runs_bytes);  // for round + 2
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[j] = after(pA[j], pb[j], state[j]);
                state[j] = after(tA[j], tb[j], state[j]);
            }
        }
        auto replay = [&](auto select, auto whole) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float out[V], dla[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const bool drop = decltype(select)::value && a[i][j] == 0.f;
                    if (BWD) {
                        // s: what the run before passed on, then the rows' dx.  The sum is one
                        // operation in both forms, so that a channel's bits do not hang on
                        // whether another one of its warp restarts.
                        const float before = i > 0 ? a[i > 0 ? i - 1 : 0][j] : 1.f;
                        s[j] = decltype(select)::value && before == 0.f ? v[i][j] : fmaf(before, s[j], v[i][j]);
                        out[j] = s[j];
                        dla[j] = drop ? 0.f : a[i][j] * s[j] * hp[BWD ? i : 0][j];
                    } else {
                        s[j] = drop ? v[i][j] : fmaf(a[i][j], s[j], v[i][j]);
                        out[j] = s[j];
                    }
                }
                if (on && (decltype(whole)::value || u0 + i < p.T)) {
                    store_row<V>(y + i * step, out);
                    if (BWD) store_row<V>(dlog_a + i * step, dla);
                }
            }
        };
        if (cut || u0 + R > p.T) replay(std::true_type(), std::false_type());
        else replay(std::false_type(), std::true_type());
        u0 += leap;
        y += leap * step;
        if (BWD) dlog_a += leap * step;
    }
    if (n > 1) {
        cluster_barrier();  // no CTA ends while another may still write to it
        if (gave_up && threadIdx.x == 0) {
            if (p.dev_status) *p.dev_status = LA_ERR_TIMEOUT;
            // runs it did not wait for may still be on their way here: microseconds
            for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 50000;) {}
        }
    }
    if (p.s_out && on && rank == 0 && w == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.s_out[(size_t)b * p.D + c0 + j] = state[j];
    }
}

// Short walks over many channels: a thread takes two channels of a sequence from end to
// end, eight rows' loads ahead, with no exchange between threads.
template <typename T, bool BWD>
__global__ void __launch_bounds__(128) scan_short_kernel(const __grid_constant__ ScanParams p, unsigned pairs) {
    constexpr int R = 8;
    const unsigned i = blockIdx.x * 128 + threadIdx.x;
    if (i >= pairs) return;
    const unsigned half = (unsigned)p.D / 2, b = i / half;
    const long long c = (long long)b * p.D + 2 * (i - b * half);  // in [B][D]
    const long long step = BWD ? -(long long)p.D : (long long)p.D;
    const long long origin = c + (long long)b * (p.T - 1) * p.D + (BWD ? (p.T - 1ll) * p.D : 0);
    const float* log_a = p.log_a + origin;
    const T* x = (const T*)p.x + origin;
    const T* h_in = (const T*)p.h_in + origin + step;  // a token earlier
    T* y = (T*)p.y + origin;
    float* dlog_a = p.dlog_a + origin;
    float s[2] = {0.f, 0.f};
    if (p.s0) row_floats<2>(p.s0 + c, s);
    float h0[2] = {0.f, 0.f};
    if (BWD && p.h0) row_floats<2>(p.h0 + c, h0);
    struct Rows {
        float a[R][2], v[R][2], h[BWD ? R : 1][2];
    } now, next;
    const int last = p.T - 1;
    auto fetch = [&](Rows& r, int u0) {  // past the end the last row again: no branch holds a load back
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const long long at = min(u0 + k, last) * step;
            row_floats<2>(log_a + at, r.a[k]);
            row_floats<2>(x + at, r.v[k]);
            if (BWD) row_floats<2>(h_in + min(u0 + k, last - 1) * step, r.h[BWD ? k : 0]);  // T = 1: token 0, unused
        }
    };
    auto work = [&](const Rows& r, int u0) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (u0 + k > last) break;
            float out[2], dla[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float a = expf(r.a[k][j]);
                if (BWD) {
                    const float h = u0 + k == last ? h0[j] : r.h[BWD ? k : 0][j];
                    out[j] = r.v[k][j] + s[j];
                    s[j] = a == 0.f ? 0.f : a * out[j];
                    dla[j] = a == 0.f ? 0.f : s[j] * h;
                } else {
                    s[j] = out[j] = after(a, r.v[k][j], s[j]);
                }
            }
            store_row<2>(y + (u0 + k) * step, out);
            if (BWD) store_row<2>(dlog_a + (u0 + k) * step, dla);
        }
    };
    fetch(now, 0);
    for (int u0 = 0; u0 < p.T; u0 += 2 * R) {
        fetch(next, u0 + R);
        work(now, u0);
        fetch(now, u0 + 2 * R);
        work(next, u0 + R);
    }
    if (p.s_out) store_row<2>(p.s_out + c, s);
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

template <typename K>
cudaError_t launch_kernel(const ScanParams& p, int B, int cluster, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(scan_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)K::kShared);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)B * p.tiles * cluster));
    cfg.blockDim = dim3(K::W * 32);
    cfg.dynamicSmemBytes = K::kShared;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TraceScope trace(K::BWD ? "scan_bwd_kernel" : "scan_kernel", s);
    return cudaLaunchKernelEx(&cfg, scan_kernel<K>, p);
}

template <typename K>
cudaError_t launch(ScanParams p, int B, int cluster, cudaStream_t s) {
    p.tiles = (int)((p.D + (K::C - 1ll)) / K::C);  // D may be 2^31 - 16
    p.mute = opt_force_timeout();
    p.limit_ns = p.mute ? 1000000ull : 2000000000ull;
    return launch_kernel<K>(p, B, cluster, s);
}

// How well `ctas` CTAs, four of which fit an SM, use the card: their spread over the
// SMs, at least 1.6 an SM needed to keep the memory busy, less for the exchange in
// clusters.  More waves spread themselves out, by and by.  Within 0.1 of the fractions of
// the copy rate measured at 97 to 400 tiles of 8192 tokens.
double card_use(long long ctas, int cluster, long long sms) {
    const double exchange = cluster == 8 ? 0.75 : cluster > 1 ? 0.93 : 1.0;
    const double per_sm = (double)ctas / (double)sms, waves = per_sm / 4;
    if (waves > 1) return (0.35 + 0.65 * waves / std::ceil(waves)) * exchange;
    return per_sm / std::ceil(per_sm) * std::min(1.0, per_sm / 1.6) * exchange;
}

// The shape and the cluster, by the channel tiles there are (fractions of the copy rate,
// one GB300, bf16, 8192 tokens unless said).  CTAs of four warps, four on an SM, out of step
// with each other, in the clusters that use the card best (97 tiles of 32 channels in
// fours 0.69, 195 in twos 0.78, 256 uncut 0.85, 1024 in fours 0.90 to 0.97); a long walk of
// more than a wave is cut in four.  Where no cluster fills the card the walk waits for its
// rounds: larger CTAs then make fewer, of six warps forward in bf16 where clusters of
// eight give every SM one (19 tiles and more; 1 x 65536 x 1024: 0.74 with six warps, 0.66
// with eight, 0.67 with four; 32 tiles of 16384 tokens 35 us with six, 38 with eight; 16 to
// 19 tiles of 65536 tokens within 2 %), of eight below (12 tiles of 65536 tokens 72 us with
// eight, 79 with six; 1 x 55483 x 256: 0.26 with eight, 0.20 with four).
//
// Backward in bf16, where tiles of 64 channels are 0.72 to 0.86 of a wave of one CTA an SM,
// two channels a lane (us, against one channel a lane, at 4096 / 8192 / 32768 tokens):
//   100 tiles 74 (66) / 140 (138) / 536 (570)    110 tiles 74 (74) / 140 (156) / 537 (622)
//   121 tiles 74 (83) / 141 (161) / 537 (660)    128 tiles 74 (79) / 140 (150) / 537 (585)
//   132 tiles 77 (81) / 155 (152) / 656 (597)    136 tiles 86 (82) / 173 (156) / 690 (603)
//   152 tiles 103 (88) / 201 (170) / 775 (728)
template <typename T, bool BWD>
cudaError_t launch(const ScanParams& p, int B, cudaStream_t s) {
    constexpr int R = BWD ? 16 : 64 / (int)sizeof(T);  // backward three tensors' rows are in registers
    using Small = Shape<T, 1, R, 4, 2, 4, BWD>;
    using Large = Shape<T, 1, R, 8, 2, 2, BWD>;
    const long long sms = sm_count(), tiles = (p.D + 31ll) / 32 * B, channels = (long long)B * p.D;
    // us at 262,144 channels: 16 tokens 12 (a round of the ring 49), 64 tokens 30 (53), 128
    // tokens 53 (57); at 1024 channels 16 tokens 8 either way, 64 tokens 12 (8)
    if ((p.T <= 16 || (p.T <= 64 && p.T * 2048ll <= channels)) && channels < 1ll << 31) {
        const unsigned pairs = (unsigned)(channels / 2);
        TraceScope trace(BWD ? "scan_short_bwd_kernel" : "scan_short_kernel", s);
        scan_short_kernel<T, BWD><<<(pairs + 127) / 128, 128, 0, s>>>(p, pairs);
        return cudaGetLastError();
    }
    if constexpr (BWD && sizeof(T) == 2) {
        const long long wide = (p.D + 63ll) / 64 * B;
        if (wide * 100 >= sms * 72 && wide * 100 <= sms * 86)
            return launch<Shape<T, 2, 16, 8, 2, 1, true>>(p, B, 1, s);
    }
    if (tiles > 4 * sms)
        return launch<Small>(p, B, tiles < 16 * sms && p.T >= 16 * Small::kRun ? 4 : 1, s);
    int cluster = 1;
    double use = card_use(tiles, 1, sms);
    for (int c = 2; c <= kMaxCluster && (long long)(c / 2) * Small::kRun < p.T; c *= 2)
        if (card_use(tiles * c, c, sms) > use) cluster = c, use = card_use(tiles * c, c, sms);
    if (use >= 0.65 || p.T <= Small::kRun) return launch<Small>(p, B, cluster, s);
    cluster = 1;
    while (cluster < kMaxCluster && tiles * cluster <= sms && (long long)cluster * Large::kRun < p.T)
        cluster *= 2;
    if constexpr (!BWD && sizeof(T) == 2)
        if (tiles * kMaxCluster >= sms) return launch<Shape<T, 1, R, 6, 2, 2, BWD>>(p, B, cluster, s);
    return launch<Large>(p, B, cluster, s);
}

}  // namespace

cudaError_t launch_scan_fwd(const RecurrenceArgs& a, cudaStream_t s) {
    ScanParams p = {};
    p.x = a.x; p.log_a = a.log_a; p.s0 = a.h0; p.y = a.h; p.s_out = a.h_out;
    p.T = a.T; p.D = a.D; p.dev_status = a.dev_status;
    const cudaError_t e = a.bf16 ? launch<__nv_bfloat16, false>(p, a.B, s)
                                 : launch<float, false>(p, a.B, s);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_scan_bwd(const RecurrenceArgs& a, cudaStream_t s) {
    ScanParams p = {};
    p.x = a.dh; p.log_a = a.log_a; p.s0 = a.dh_T; p.h_in = a.h; p.h0 = a.h0;
    p.y = a.dx; p.dlog_a = a.dlog_a; p.s_out = a.dh0;
    p.T = a.T; p.D = a.D; p.dev_status = a.dev_status;
    const cudaError_t e = a.bf16 ? launch<__nv_bfloat16, true>(p, a.B, s)
                                 : launch<float, true>(p, a.B, s);
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
