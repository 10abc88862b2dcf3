// The seam between two blocks of a residual stream, row by row of [B][T][D]:
//
//   p  = o  or  norm(o) w_post        (the norm after the block)
//   h' = beta h + alpha g p           (its gate, a row for all or for each sequence)
//   y  = norm(h') w_pre               (the norm before the next block)
//
//   norm(v) = (v - mean v) r, r = (mean (v - mean v)^2 + eps)^(-1/2)   (no mean taken
//                                                                  out unless centred)
//
// and its gradients, with dt = dh' + norm'(dy w_pre):
//
//   dh = beta dt,  dg = alpha sum p dt,  dw_pre = sum dy norm(h'),
//   do = norm'(alpha g dt w_post),  dw_post = sum alpha g dt norm(o),
//   norm'(v) = r (v - [mean v] - n mean(v n))
//
// Bound by HBM: o and h in, h' and y out; 8 x 8192 rows of 2048 in bf16 take 166 us, 0.96 of the copy
// rate, gradients of 4 x 4093 rows of 2048 (fp32 residual, centred) 103 us, 0.87, and their sums 8.  A CTA
// holds a row in registers (a thread eight neighbouring entries, once or twice), so that both norms cost no
// second read, and the weights of its columns.  The next row comes through a ring in shared memory, copied in
// the background, each thread's own pieces (fp32: each warp's).  Rows are dealt out to the CTAs in turn: a run
// of rows for each took 200 us where this takes 190.  Rows that fill their threads have a build without
// questions after single entries (the gradients 113 us without, 103 with).  dg and dw_post are one sum over
// the rows, of alpha dt p, times w_post and g.  y is the norm of h' before its rounding; the gradients start
// from the rounded h' that the forward call left.
#include <algorithm>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

struct Rows {
    const void* p;
    long long b, t;  // strides
    bool wide;       // rows of fp32 start at multiples of 32 bytes
};

struct BlockParams {
    Rows o, h, dy, dh;             // h: the residual, backward h'; null pointers where absent
    Rows h_out, y, d_o, d_res;     // outputs
    const float *w_post, *gate, *w_pre;
    float *part_post, *part_gate, *part_pre;  // backward: partial rows, or null
    int B, T, D;
    int rows_cta;                  // rows a CTA holds at once
    int ring;                      // backward: rows of the ring in shared memory
    Divide by_T;
    int seq_blocks;                // CTAs a sequence's rows are shared out to (0: of all sequences)
    int post, pre, center, gate_each;
    float alpha, beta, eps;
};

// Sums of N values over the threads of a row, in a fixed order.  `red`: [2][N][16] floats of
// the row's slot, its halves in turn, so that one barrier a sum is enough; what a row has fewer than
// 16 warps is zero from the start.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& turn, int warps, int warp) {
    const int lane = threadIdx.x & 31;
    float* to = red + turn * 32;
    if (N == 1) {
        v[0] = group_sum<32>(v[0]);
        if (warps == 1) return;
        if (lane == 0) to[warp] = v[0];
    } else {  // the lower half of the warp takes the first value, the upper half the second
        const bool hi = lane & 16;
        const float keep = hi ? v[N - 1] : v[0], send = hi ? v[0] : v[N - 1];
        const float sum = group_sum<16>(keep + __shfl_xor_sync(0xffffffffu, send, 16));
        if (warps == 1) {
            v[0] = __shfl_sync(0xffffffffu, sum, 0);
            v[N - 1] = __shfl_sync(0xffffffffu, sum, 16);
            return;
        }
        if ((lane & 15) == 0) to[lane + warp] = sum;
    }
    turn ^= 1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float4* from = reinterpret_cast<const float4*>(to + i * 16);
        float4 s = from[0];
        for (int k = 1; k * 4 < warps; ++k) {
            const float4 r = from[k];
            s.x += r.x; s.y += r.y; s.z += r.z; s.w += r.w;
        }
        v[i] = (s.x + s.y) + (s.z + s.w);
    }
}

// Two rows' slots at most share a CTA's barriers; one value's sum uses the first half's 16.
constexpr int kRedFloats = 2 * 2 * 16;

__device__ __forceinline__ void clear_red(float (*red)[kRedFloats], int slots) {
    for (int i = threadIdx.x; i < slots * kRedFloats; i += blockDim.x) red[0][i] = 0.f;
    __syncthreads();
}

__device__ __forceinline__ float sum8(const float2 (&x)[4]) {
    const float2 s = __fadd2_rn(__fadd2_rn(x[0], x[1]), __fadd2_rn(x[2], x[3]));
    return s.x + s.y;
}

// A thread's place: row slot, its warp in the row, its first entry.
struct Place {
    int slot, warp, warps, lane;
    // one row a CTA: slot 0 known to all, so that its rows' addresses are the CTA's, not each thread's
    __device__ Place(int rows_cta, bool one) {
        const int per = one ? blockDim.x : blockDim.x / rows_cta;
        slot = one ? 0 : threadIdx.x / per;
        lane = threadIdx.x - slot * per;
        warps = per / 32;
        warp = lane / 32;
    }
};

// A row's place, walking by a fixed number of rows.
struct Walk {
    unsigned b, t, leap_b, leap_t, T;
    __device__ Walk(const Divide& by_T, unsigned row, unsigned leap) : T(by_T.T) {
        by_T(row, &b, &t);
        by_T(leap, &leap_b, &leap_t);
    }
    __device__ __forceinline__ void next() {
        b += leap_b;
        t += leap_t;
        if (t >= T) t -= T, ++b;
    }
    template <typename E>
    __device__ __forceinline__ E* at(const Rows& r) const {
        return (E*)r.p + b * r.b + t * r.t;
    }
};

// A thread's eight entries from e on into its slot in the background.  fp32 entries a warp copies
// together, 512 bytes in a row at once (a thread's own 32 bytes are two halves of a sector, fetched twice).
// Their pieces of four lie exchanged in every second group of four lanes, which then read without a
// bank met twice.
template <bool WHOLE, typename E>
__device__ __forceinline__ void copy8(E* slot, const E* row, int e, int D) {
    if constexpr (sizeof(E) == 2) {
        if (WHOLE || e < D) copy16(slot, row + e, true);
    } else {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int q = k * 32 + lane;
            if (WHOLE || e - lane * 8 + q * 4 < D)
                copy16(slot - lane * 8 + (q ^ (q >> 3 & 1)) * 4, row + e - lane * 8 + q * 4, true);
        }
    }
}

template <typename E>
__device__ __forceinline__ void read8(const E* slot, float2 (&x)[4]) {
    const int s = sizeof(E) == 2 ? 0 : threadIdx.x >> 2 & 1;
    floats8<false>(raw8<sizeof(E) == 2>(slot, 4 * s, 4 - 4 * s), x);
}

// Around a warp's reads of what its lanes copied for one another.
template <typename T, typename R>
__device__ __forceinline__ void warp_slots() {
    if constexpr (sizeof(T) == 4 || sizeof(R) == 4) __syncwarp();
}

// Eight entries to memory: fp32 ones in one 32-byte access where every row allows it.
template <typename E>
__device__ __forceinline__ void put8(E* to, const float2 (&x)[4], bool wide) {
    if constexpr (sizeof(E) == 4) {
        if (wide) {
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(x[0].x), "f"(x[0].y),
                         "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y)
                         : "memory");
            return;
        }
    }
    store8<true, false>(to, 0, 4, x);
}

template <bool MINUS_MEAN, int P>
__device__ __forceinline__ float normed(float2 (&x)[P][4], const bool (&on)[P], float inv_d, float eps, float* red,
                                        int& turn, const Place& at) {
    if (MINUS_MEAN) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) s[0] += sum8(x[i]);
        row_sums<1>(s, red, turn, at.warps, at.warp);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (on[i])
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = __fadd2_rn(x[i][j], both(-s[0] * inv_d));
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < P; ++i) q[0] += dot8(x[i], x[i]);
    row_sums<1>(q, red, turn, at.warps, at.warp);
    return rsqrtf(q[0] * inv_d + eps);
}

// Rows of the forward ring, by a CTA's threads: one row ahead where an SM holds three CTAs or more, whose
// rows then keep the memory busy and no more than that (8 x 8192 rows of 2048: 192 us with three rows ahead,
// 166 with one; rows of 512 to 4096 entries in bf16 0.80 of the copy rate against 0.86 to 0.93); the one
// CTA of 512 threads reaches 0.83 with three and 0.58 with one.
constexpr int fwd_ring(int threads) { return threads > 256 ? 3 : 1; }

// T: o and y; R: the residual stream.  P pieces of eight entries a thread.
template <typename T, typename R, int P, int THREADS, bool CENTER, bool WHOLE>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 1 : 768 / THREADS)
    block_norm_kernel(const __grid_constant__ BlockParams p) {
    __shared__ __align__(16) float red[4][kRedFloats];
    clear_red(red, 4);
    constexpr int kRing = fwd_ring(THREADS);
    extern __shared__ __align__(16) unsigned char ring[];  // [kRing][P][threads] of T's eight, then of R's
    const Place at(p.rows_cta, WHOLE);
    const int width = at.warps * 32 * 8;  // entries of a piece of the row
    const unsigned rows = p.by_T.T * (unsigned)p.B, leap = gridDim.x * (WHOLE ? 1 : p.rows_cta);
    const float inv_d = 1.f / (float)p.D;
    T* const slots_o = reinterpret_cast<T*>(ring) + threadIdx.x * 8;
    R* const slots_h = reinterpret_cast<R*>(ring + (size_t)kRing * P * blockDim.x * 8 * sizeof(T)) + threadIdx.x * 8;
    const int piece = blockDim.x * 8;
    int turn = 0;
    bool on[P];
    int e[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        e[i] = i * width + at.lane * 8;
        on[i] = WHOLE || e[i] < p.D;
    }
    const unsigned first = blockIdx.x * p.rows_cta + at.slot;
    Walk ahead(p.by_T, first, leap), here = ahead;
    unsigned m_ahead = first;
    auto fetch = [&](int slot) {
        if (m_ahead < rows) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                copy8<WHOLE>(slots_o + (slot * P + i) * piece, ahead.at<const T>(p.o), e[i], p.D);
                if (p.h.p) copy8<WHOLE>(slots_h + (slot * P + i) * piece, ahead.at<const R>(p.h), e[i], p.D);
            }
        }
        copies_commit();
        m_ahead += leap;
        ahead.next();
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch(i);
    float2 gw[P][4], w_pre[P][4];  // alpha g w_post, w_pre
    unsigned gate_of = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < P; ++i) row_weights<false>(p.w_pre, on[i], e[i], e[i] + 4, w_pre[i]);
    int slot = 0;
    for (unsigned m = first; (WHOLE ? m : m - at.slot) < rows; m += leap) {  // the same for every slot
        const bool row = WHOLE || m < rows;
        const unsigned gate_now = p.gate_each && row ? here.b : 0;
        if (gate_now != gate_of) {
            gate_of = gate_now;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 g[4];
                row_weights<false>(p.w_post, on[i], e[i], e[i] + 4, gw[i]);
                row_weights<false>(p.gate ? p.gate + (size_t)gate_of * p.D : nullptr, on[i], e[i], e[i] + 4, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) gw[i][j] = __fmul2_rn(gw[i][j], __fmul2_rn(g[j], both(p.alpha)));
            }
        }
        float2 v[P][4];
        copies_wait<kRing - 1>();
        warp_slots<T, R>();
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = make_float2(0.f, 0.f);
            if (row && on[i]) read8(slots_o + (slot * P + i) * piece, v[i]);
        }
        float r = 1.f;
        if (p.post) r = normed<CENTER, P>(v, on, inv_d, p.eps, red[at.slot], turn, at);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 h[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
            if (row && on[i] && p.h.p) read8(slots_h + (slot * P + i) * piece, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = __fmul2_rn(__fmul2_rn(v[i][j], both(r)), gw[i][j]);
                v[i][j] = __ffma2_rn(h[j], both(p.beta), v[i][j]);
            }
            if (row && on[i] && p.h_out.p) put8(here.at<R>(p.h_out) + e[i], v[i], p.h_out.wide);
        }
        warp_slots<T, R>();
        fetch(slot);
        slot = slot + 1 == kRing ? 0 : slot + 1;
        if (p.pre) {
            r = normed<CENTER, P>(v, on, inv_d, p.eps, red[at.slot], turn, at);
#pragma unroll
            for (int i = 0; i < P; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(__fmul2_rn(v[i][j], both(r)), w_pre[i][j]);
                if (row && on[i]) put8(here.at<T>(p.y) + e[i], v[i], p.y.wide);
            }
        }
        here.next();
    }
}

// A CTA takes rows of one sequence where each sequence has its own gate (its sums then
// belong to that sequence's gradient), else of all.
template <typename T, typename R, int P, int THREADS, bool CENTER, bool WHOLE>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) block_norm_bwd_kernel(const __grid_constant__ BlockParams p) {
    tc::griddep_launch_dependents();  // the sums' kernel may be scheduled (it waits itself)
    __shared__ __align__(16) float red[4][kRedFloats];
    clear_red(red, 4);
    extern __shared__ __align__(16) unsigned char ring[];  // o, dy, h, dh; at the end [rows_cta][D] sums
    const Place at(p.rows_cta, WHOLE);
    const int width = at.warps * 32 * 8;
    const unsigned begin = p.seq_blocks ? blockIdx.x / p.seq_blocks * p.by_T.T : 0;
    const unsigned end = p.seq_blocks ? begin + p.by_T.T : p.by_T.T * (unsigned)p.B;
    const unsigned leap = (p.seq_blocks ? p.seq_blocks : gridDim.x) * p.rows_cta;
    const unsigned first = begin + (p.seq_blocks ? blockIdx.x % p.seq_blocks : blockIdx.x) * p.rows_cta + at.slot;
    const float inv_d = 1.f / (float)p.D;
    const int piece = blockDim.x * 8;
    T* const slots_t = reinterpret_cast<T*>(ring) + threadIdx.x * 8;  // [p.ring][2][P]
    R* const slots_r = reinterpret_cast<R*>(ring + (size_t)p.ring * 2 * P * piece * sizeof(T)) + threadIdx.x * 8;
    int turn = 0;
    bool on[P];
    int e[P];
    float2 s_post[P][4], s_pre[P][4];  // sums of alpha dt p and dy n
    const float* gate = p.gate ? p.gate + (p.seq_blocks ? (size_t)(blockIdx.x / p.seq_blocks) * p.D : 0) : nullptr;
    // the thread's entries of alpha g w_post and of w_pre, in shared memory: two quads of each
    float4* const gws = reinterpret_cast<float4*>(reinterpret_cast<R*>(ring + (size_t)p.ring * 2 * P * piece * sizeof(T)) +
                                                  (size_t)p.ring * 2 * P * piece) + threadIdx.x;
    float4* const w_pres = gws + 2 * P * blockDim.x;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        e[i] = i * width + at.lane * 8;
        on[i] = WHOLE || e[i] < p.D;
#pragma unroll
        for (int j = 0; j < 4; ++j) s_post[i][j] = s_pre[i][j] = make_float2(0.f, 0.f);
    }
    Walk ahead(p.by_T, first, leap), here = ahead;
    unsigned m_ahead = first;
    auto fetch = [&](int slot) {
        if (m_ahead < end) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                T* const t = slots_t + (slot * 2 * P + i) * piece;
                R* const r = slots_r + (slot * 2 * P + i) * piece;
                copy8<WHOLE>(t, ahead.at<const T>(p.o), e[i], p.D);
                if (p.pre) {
                    copy8<WHOLE>(t + P * piece, ahead.at<const T>(p.dy), e[i], p.D);
                    copy8<WHOLE>(r, ahead.at<const R>(p.h), e[i], p.D);
                }
                if (p.dh.p) copy8<WHOLE>(r + P * piece, ahead.at<const R>(p.dh), e[i], p.D);
            }
        }
        copies_commit();
        m_ahead += leap;
        ahead.next();
    };
    for (int i = 0; i < p.ring; ++i) fetch(i);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float2 g[4], w[4];
        row_weights<false>(p.w_post, on[i], e[i], e[i] + 4, w);
        row_weights<false>(gate, on[i], e[i], e[i] + 4, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(w[j], __fmul2_rn(g[j], both(p.alpha)));
        row_weights<false>(p.w_pre, on[i], e[i], e[i] + 4, w);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            gws[(2 * i + k) * blockDim.x] = make_float4(g[2 * k].x, g[2 * k].y, g[2 * k + 1].x, g[2 * k + 1].y);
            w_pres[(2 * i + k) * blockDim.x] = make_float4(w[2 * k].x, w[2 * k].y, w[2 * k + 1].x, w[2 * k + 1].y);
        }
    }
    auto weights = [&](const float4* from, int i, float2 (&w)[4]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 f = from[(2 * i + k) * blockDim.x];
            w[2 * k] = make_float2(f.x, f.y);
            w[2 * k + 1] = make_float2(f.z, f.w);
        }
    };
    int slot = 0;
    for (unsigned m = first; (WHOLE ? m : m - at.slot) < end; m += leap) {
        const bool row = WHOLE || m < end;
        float2 n[P][4], q[P][4], dt[P][4];  // norm(h'), p, and dy on its way to dt
        if (p.ring == 1) copies_wait<0>();
        else copies_wait<1>();
        warp_slots<T, R>();
        auto take = [&](auto* slots, int which, int i, float2 (&to)[4]) {  // zeros where there is nothing
            if (row && on[i]) {
                read8(slots + (slot * 2 * P + which * P + i) * piece, to);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) to[j] = make_float2(0.f, 0.f);
            }
        };
        // both rows' norms: means, then squares
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            take(slots_t, 0, i, q[i]);
            if (p.pre) {
                take(slots_r, 0, i, n[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) n[i][j] = make_float2(0.f, 0.f);
            }
        }
        if (CENTER) {
#pragma unroll
            for (int i = 0; i < P; ++i) s[0] += sum8(n[i]), s[1] += sum8(q[i]);
            row_sums<2>(s, red[at.slot], turn, at.warps, at.warp);
            const float2 mh = both(-s[0] * inv_d), mo = both(p.post ? -s[1] * inv_d : 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (on[i])
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        n[i][j] = __fadd2_rn(n[i][j], mh);
                        q[i][j] = __fadd2_rn(q[i][j], mo);
                    }
            s[0] = s[1] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) s[0] += dot8(n[i], n[i]), s[1] += dot8(q[i], q[i]);
        row_sums<2>(s, red[at.slot], turn, at.warps, at.warp);
        const float rh = rsqrtf(s[0] * inv_d + p.eps), ro = p.post ? rsqrtf(s[1] * inv_d + p.eps) : 1.f;
        if (p.pre) {
            s[0] = s[1] = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 w[4];
                __syncwarp();
                take(slots_t, 1, i, dt[i]);
                weights(w_pres, i, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[i][j] = __fmul2_rn(n[i][j], both(rh));
                    s_pre[i][j] = __ffma2_rn(dt[i][j], n[i][j], s_pre[i][j]);
                    dt[i][j] = __fmul2_rn(dt[i][j], w[j]);
                }
                s[0] += dot8(dt[i], n[i]);
                if (CENTER) s[1] += sum8(dt[i]);
            }
            row_sums<2>(s, red[at.slot], turn, at.warps, at.warp);
        }
        const float2 along_h = both(-s[0] * inv_d), mean_h = both(CENTER ? -s[1] * inv_d : 0.f);
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 into[4], w[4];
            if (p.dh.p) {
                __syncwarp();
                take(slots_r, 1, i, into);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) into[j] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p.pre && on[i])
                    into[j] = __ffma2_rn(both(rh), __ffma2_rn(n[i][j], along_h, __fadd2_rn(dt[i][j], mean_h)), into[j]);
                dt[i][j] = into[j];
            }
            if (row && on[i] && p.d_res.p) {
#pragma unroll
                for (int j = 0; j < 4; ++j) into[j] = __fmul2_rn(into[j], both(p.beta));
                put8(here.at<R>(p.d_res) + e[i], into, p.d_res.wide);
            }
            weights(gws, i, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[i][j] = __fmul2_rn(q[i][j], both(ro));
                s_post[i][j] = __ffma2_rn(__fmul2_rn(dt[i][j], both(p.alpha)), q[i][j], s_post[i][j]);
                dt[i][j] = __fmul2_rn(dt[i][j], w[j]);
            }
            s[0] += dot8(dt[i], q[i]);
            if (CENTER) s[1] += sum8(dt[i]);
        }
        warp_slots<T, R>();
        fetch(slot);
        slot = slot + 1 == p.ring ? 0 : slot + 1;
        if (p.post) {
            row_sums<2>(s, red[at.slot], turn, at.warps, at.warp);
            const float2 along = both(-s[0] * inv_d), mean = both(CENTER ? -s[1] * inv_d : 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dt[i][j] = __fmul2_rn(both(ro), __ffma2_rn(q[i][j], along, __fadd2_rn(dt[i][j], mean)));
        }
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (row && on[i]) put8(here.at<T>(p.d_o) + e[i], dt[i], p.d_o.wide);
        here.next();
    }
    // one partial row a CTA, over its row slots
    copies_wait<0>();
    float* const columns = reinterpret_cast<float*>(ring);
    auto leave = [&](const float2 (&sum)[P][4], const float* times, float* part) {
        if (!part) return;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (on[i]) {
                float2 f[4];
                row_weights<false>(times, on[i], e[i], e[i] + 4, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(f[j], sum[i][j]);
                store8<true, false>(columns + (size_t)at.slot * p.D + e[i], 0, 4, f);
            }
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            float v = 0.f;
            for (int k = 0; k < p.rows_cta; ++k) v += columns[(size_t)k * p.D + c];
            part[(size_t)blockIdx.x * p.D + c] = v;
        }
    };
    leave(s_post, gate, p.part_post);
    leave(s_post, p.w_post, p.part_gate);
    leave(s_pre, nullptr, p.part_pre);
}

// d(gate) of each sequence: its CTAs' partial rows, added in order.
__global__ void __launch_bounds__(128) block_gate_sum_kernel(const float* part, int blocks, int D, float* out) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= D) return;
    const float* from = part + (size_t)blockIdx.y * blocks * D + c;
    float v = 0.f;
    for (int k = 0; k < blocks; ++k) v += from[(size_t)k * D];
    out[(size_t)blockIdx.y * D + c] = v;
}

struct Shape {
    int pieces, threads, rows;  // a row's pieces a thread and threads, rows a CTA
};

// Two pieces a thread above 256 entries: fewer warps a row, whose sums cost less.  A row just above a
// multiple of 512 entries leaves up to half of its threads without any, which shows in bf16 (of the
// copy rate, forward and gradients: 512 entries 0.88 and 0.84, 528 0.59 and 0.44, 768 0.75 and 0.63, 1024 0.84 and
// 0.78, 1040 0.69 and 0.52, 1536 0.90 and 0.88; fp32 0.86 to 0.96 and 0.76 to 0.95).
Shape shape(int D) {
    Shape s;
    s.pieces = D <= 256 ? 1 : 2;
    const int per = 8 * s.pieces;
    s.threads = ((D + per - 1) / per + 31) / 32 * 32;
    s.rows = s.threads <= 32 ? 4 : s.threads <= 64 ? 2 : 1;
    return s;
}

// Bytes of a CTA's shared memory, T and R the sizes of an entry of o and of the residual.
size_t fwd_shared(const Shape& sh, size_t T, size_t R) {
    const size_t entries = (size_t)sh.pieces * sh.threads * sh.rows * 8;
    return entries * fwd_ring(sh.threads * sh.rows) * (T + R);
}
size_t bwd_shared(const Shape& sh, size_t T, size_t R, int ring) {
    const size_t entries = (size_t)sh.pieces * sh.threads * sh.rows * 8;
    return entries * (ring * 2 * (T + R) + 2 * sizeof(float));  // the sums at the end fit in the ring
}

constexpr size_t kMostShared = 222 << 10;  // of a CTA, beside its static part

// CTAs an SM holds: by the registers the launch bounds leave a thread, and by shared memory.
long long resident(const Shape& sh, int threads_per_sm, size_t shared) {
    const long long by_threads = threads_per_sm / (sh.threads * sh.rows);
    const long long by_shared = (long long)((224u << 10) / (shared + 2048));
    return std::max(1ll, std::min(by_threads, by_shared));
}

size_t entry_size(bool bf16) { return bf16 ? 2 : 4; }

// Rows of the gradients' ring: two where the second costs an SM no CTA (rows of 2048 in bf16 0.89 of the copy rate,
// with one row 0.83; 5120 0.59 and 0.49), else one (2048 beside an fp32 residual 0.96, with two rows and a CTA
// fewer 0.84; 4096 in bf16 0.77 and 0.60).
int bwd_ring(const Shape& sh, size_t T, size_t R) {
    const size_t two = bwd_shared(sh, T, R, 2);
    return two <= kMostShared && resident(sh, 512, two) == resident(sh, 512, bwd_shared(sh, T, R, 1)) ? 2 : 1;
}

long long fwd_blocks(const BlockNormArgs& a) {
    const Shape sh = shape(a.D);
    const long long rows = ((long long)a.B * a.T + sh.rows - 1) / sh.rows;
    const size_t shared = fwd_shared(sh, entry_size(a.bf16), entry_size(a.residual_bf16));
    return std::min(rows, sm_count() * resident(sh, sh.threads > 256 ? 512 : 768, shared));
}

// CTAs of the gradients: (of each sequence, in all).
void bwd_blocks(const BlockNormArgs& a, int* each, long long* all) {
    const Shape sh = shape(a.D);
    // as many for either type of the residual: the workspace's size is asked for without it
    const size_t entry = entry_size(a.bf16);
    const long long most = sm_count() * resident(sh, 512, bwd_shared(sh, entry, 4, bwd_ring(sh, entry, 4)));
    if (a.gate && a.gate_each) {
        const long long rows = ((long long)a.T + sh.rows - 1) / sh.rows;
        *each = (int)std::max(1ll, std::min(rows, most / a.B));
        *all = (long long)*each * a.B;
    } else {
        *each = 0;
        *all = std::min(((long long)a.B * a.T + sh.rows - 1) / sh.rows, most);
    }
}

BlockParams params(const BlockNormArgs& a) {
    auto rows = [](const void* p, const long long* s) {
        return Rows{p, s[0], s[1], (reinterpret_cast<uintptr_t>(p) | s[0] * 4 | s[1] * 4) % 32 == 0};
    };
    BlockParams p = {};
    p.o = rows(a.o, a.o_strides);
    p.h = rows(a.h, a.h_strides);
    p.dy = rows(a.dy, a.dy_strides);
    p.dh = rows(a.dh, a.dh_strides);
    p.h_out = rows(a.h_out, a.h_out_strides);
    p.y = rows(a.y, a.y_strides);
    p.d_o = rows(a.d_o, a.d_o_strides);
    p.d_res = rows(a.d_res, a.d_res_strides);
    p.w_post = a.post_weight; p.gate = a.gate; p.w_pre = a.pre_weight;
    p.B = a.B; p.T = a.T; p.D = a.D;
    p.rows_cta = shape(a.D).rows;
    p.by_T = Divide::by(a.T);
    p.post = a.post; p.pre = a.pre; p.center = a.center; p.gate_each = a.gate_each;
    p.alpha = a.scale; p.beta = a.residual_scale; p.eps = a.eps;
    return p;
}

template <typename T, typename R, int P, int THREADS, bool CENTER, bool WHOLE>
cudaError_t launch(const BlockParams& p, bool bwd, unsigned grid, int threads, cudaStream_t s) {
    const Shape sh = shape(p.D);
    const size_t shared = bwd ? bwd_shared(sh, sizeof(T), sizeof(R), p.ring) : fwd_shared(sh, sizeof(T), sizeof(R));
    const auto kernel = bwd ? block_norm_bwd_kernel<T, R, P, THREADS, CENTER, WHOLE>
                            : block_norm_kernel<T, R, P, THREADS, CENTER, WHOLE>;
    if (shared > 44 * 1024) {  // less, with the static part, a kernel has without asking
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, threads, shared, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename R, int P, int THREADS>
cudaError_t launch(const BlockParams& p, bool bwd, unsigned grid, int threads, cudaStream_t s) {
    // a row for the CTA's threads, none of them past its end: no entry needs asking for
    if constexpr (P > 1) {
        if (p.rows_cta == 1 && p.D == 8 * P * threads)
            return p.center ? launch<T, R, P, THREADS, true, true>(p, bwd, grid, threads, s)
                            : launch<T, R, P, THREADS, false, true>(p, bwd, grid, threads, s);
    }
    return p.center ? launch<T, R, P, THREADS, true, false>(p, bwd, grid, threads, s)
                    : launch<T, R, P, THREADS, false, false>(p, bwd, grid, threads, s);
}

template <typename T, typename R>
cudaError_t launch(const BlockParams& p, bool bwd, unsigned grid, cudaStream_t s) {
    const Shape sh = shape(p.D);
    const int threads = sh.threads * sh.rows;
    if (sh.pieces == 1) return launch<T, R, 1, 128>(p, bwd, grid, threads, s);
    if (threads <= 256) return launch<T, R, 2, 256>(p, bwd, grid, threads, s);
    return launch<T, R, 2, 512>(p, bwd, grid, threads, s);
}

cudaError_t launch(const BlockNormArgs& a, const BlockParams& p, bool bwd, unsigned grid, cudaStream_t s) {
    if (!a.bf16) return launch<float, float>(p, bwd, grid, s);
    if (a.residual_bf16) return launch<__nv_bfloat16, __nv_bfloat16>(p, bwd, grid, s);
    return launch<__nv_bfloat16, float>(p, bwd, grid, s);
}

}  // namespace

size_t block_norm_bwd_workspace_bytes(const BlockNormArgs& a) {
    int each;
    long long all;
    bwd_blocks(a, &each, &all);
    return (size_t)all * a.D * 3 * sizeof(float);
}

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, cudaStream_t s) {
    TraceScope trace("block_norm_kernel", s);
    return launch(a, params(a), false, (unsigned)fwd_blocks(a), s);
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, cudaStream_t s) {
    BlockParams p = params(a);
    p.ring = bwd_ring(shape(a.D), entry_size(a.bf16), entry_size(a.residual_bf16));
    int each;
    long long all;
    bwd_blocks(a, &each, &all);
    p.seq_blocks = each;
    float* part = (float*)a.workspace;
    if (a.dpost_weight) p.part_post = part;
    if (a.dgate) p.part_gate = part + (size_t)all * a.D;
    if (a.dpre_weight) p.part_pre = part + (size_t)all * a.D * 2;
    const bool sums = p.part_post || p.part_gate || p.part_pre;
    cudaError_t e;
    {
        TraceScope trace("block_norm_bwd_kernel", s);
        e = launch(a, p, true, (unsigned)all, s);
    }
    if (e != cudaSuccess || !sums) return e;
    const PartialSum of[3] = {{p.part_post, a.dpost_weight, (int)all, a.D},
                              {p.part_gate, each ? nullptr : a.dgate, (int)all, a.D},
                              {p.part_pre, a.dpre_weight, (int)all, a.D}};
    e = launch_partial_sums(of, 3, s);
    if (e != cudaSuccess || !each || !a.dgate) return e;
    TraceScope trace("block_gate_sum_kernel", s);
    block_gate_sum_kernel<<<dim3((a.D + 127) / 128, a.B), 128, 0, s>>>(p.part_gate, each, a.D, a.dgate);
    return cudaGetLastError();
}

}  // namespace la
