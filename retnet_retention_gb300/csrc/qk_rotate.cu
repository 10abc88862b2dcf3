// Queries and keys made ready for retention in one pass: the norm of each head's
// row, the rotation by its token's position, a scale, and the change of layout
// from the projections' [B][T][H][d] (any strides) to [B][H][T][d].
//
//   n = x r w,  r = (mean(x^2) + eps)^(-1/2)                 (x itself without the norm)
//   y1 = s (n1 cos - n2 sin),  y2 = s (n1 sin + n2 cos)      for each pair of the first rot entries
//   y = s n                                                  for the rest
//
// and its gradient: with g = s R^T dy, dw = sum g x r over the tokens and heads,
// gx = g w and dx = r (gx - x r^2 mean(gx x)).
//
// The angle of pair i at position p is p f_i.  Its fraction of a turn is taken in
// integers: F_i = f_i / 2 pi modulo one turn, in units of 2^-64 turns, p F_i mod 2^64 is
// exact, so a position of any size keeps the angle to fp32 accuracy, without 64-bit floats.
//
// Bound by HBM: 2 bytes in and 2 out an entry (bf16), about 10 operations.  A
// group of d / 8 lanes holds one row.  With split halves a lane holds four entries
// of the first half and the four they pair with, so that the rotation needs no
// exchange between lanes.  A group keeps its token and walks heads, so that the four
// angles of a lane are computed once a token: forward the heads of q, then of k;
// backward those of one of the two, so that a lane keeps one set of weights and of
// their gradients' sums.  Forward the loads of four rows are in flight in registers (two:
// 187 us where four take 166); backward, with two tensors to read, they come through
// the ring of rows.cuh (register double buffers: 80 us where the ring takes 74).
//
// One GB300, bf16: 8 x 8192 tokens of 16 + 16 heads of 128 in 166 us (6.5 TB/s, 0.96 of
// a copy's rate); the gradients of 4 x 4096 of them in 69 us (5.8 TB/s; the kernel alone
// 61, the sums over its CTAs and the launch the rest).  With one or two heads the
// angles are the larger part: 16 x 8192 tokens of 1 + 1 heads of 128 in 44 us (3.0 TB/s).
#include <algorithm>
#include <cmath>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kThreads = 128;
constexpr int kFwdRows = 4;    // rows (heads) whose loads are in flight together
constexpr int kRingBytes = 8;  // backward: the ring's rows are kRingBytes / sizeof(T)

// q or k.
struct Side {
    const void* x;            // raw projection
    const void* g;            // backward: the gradient of its output [B][H][T][d]
    void* y;                  // output, or the projection's gradient
    const float* w;           // norm weights [d] or null
    float* part;              // backward: per-CTA weight gradients [CTA][d] or null
    long long x_b, x_t, x_h;  // strides, elements
    long long y_b, y_t, y_h;
    int H, hb, nhb;           // heads, heads a group walks at a stretch, such blocks of heads
    unsigned items, ctas;     // B nhb T: what the groups share out; this side's CTAs
    float scale;
};

struct QkParams {
    Side side[2];  // q's CTAs first
    const int* positions;         // [B][T] or null: pos0 + t
    Divide tokens;                // by T
    int pos0, d, rot, norm;
    bool both;                    // forward: a group takes its token's q and k
    float eps;
    uint2 freq[128];              // turns per position: x 2^-64 + y 2^-32
};

// Where a group stands: an item is a token and a block of heads of one side.
// Neighbouring groups take neighbouring tokens: their output rows touch.
struct Place {
    int b, t, h0, heads;  // heads 0: no such item (its group keeps the shuffles company)

    __device__ __forceinline__ Place(const QkParams& p, const Side& a, unsigned item) {
        const bool live = item < a.items;
        unsigned row, tt, bb, hblk = 0;
        p.tokens(live ? item : 0, &row, &tt);
        bb = row;
        if (a.nhb > 1) {
            bb = row / (unsigned)a.nhb;
            hblk = row - bb * (unsigned)a.nhb;
        }
        b = (int)bb;
        t = (int)tt;
        h0 = (int)hblk * a.hb;
        heads = live ? min(a.hb, a.H - h0) : 0;
    }
};

// cos and sin of p F, F = hi 2^-32 + lo 2^-64 turns.  Of the product modulo one turn
// the upper 32 bits are kept: the nearest quarter turn, and the rest, at most an eighth
// of a turn (pi / 4), whose sine and cosine are their Taylor series.  The first terms
// left out, x^11 / 11! and x^12 / 12!, are below 2^-29 there.
__device__ __forceinline__ void turn(int p, uint2 f, float* c, float* s) {
    // the product of p + 2^32 [p < 0] and F, less F 2^32 [p < 0]
    unsigned frac = __umulhi((unsigned)p, f.x) + (unsigned)p * f.y - (p < 0 ? f.x : 0u);
    frac += 1u << 29;
    const unsigned quarter = frac >> 30;
    const float x = (float)((int)(frac & 0x3fffffffu) - (1 << 29)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
    const float z = x * x;
    float sx = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    sx = fmaf(z, sx, 8.3333333e-3f);
    sx = fmaf(z, sx, -1.6666667e-1f);
    sx = fmaf(z * x, sx, x);
    float cx = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    cx = fmaf(z, cx, -1.3888889e-3f);
    cx = fmaf(z, cx, 4.1666667e-2f);
    cx = fmaf(z, cx, -0.5f);
    cx = fmaf(z, cx, 1.f);
    const float cc = (quarter & 1) ? sx : cx, ss = (quarter & 1) ? cx : sx;
    // quarters 1 and 2 turn the cosine's sign, 2 and 3 the sine's
    *c = __uint_as_float(__float_as_uint(cc) ^ ((quarter + 1) << 30 & 0x80000000u));
    *s = __uint_as_float(__float_as_uint(ss) ^ (quarter << 30 & 0x80000000u));
}

// A lane's entries and angles: entries e1..e1+3 and e2..e2+3; in the rotated part
// its four pairs are number 4 lane + j, (j, j + 4) of its eight with split halves
// and (2j, 2j + 1) with adjacent ones (held with the even entries first).
template <bool HALVES>
struct Lane {
    int e1, e2;
    bool on, turned;

    __device__ __forceinline__ Lane(int lane, int d, int rot) {
        turned = lane * 8 < rot;
        on = lane * 8 < d;
        e1 = HALVES && turned ? lane * 4 : lane * 8;
        e2 = HALVES && turned ? rot / 2 + lane * 4 : lane * 8 + 4;
    }

    __device__ __forceinline__ void angles(const uint2* freq, int lane, int pos,
                                           float2 (&c)[2], float2 (&s)[2]) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            c[j] = make_float2(1.f, 1.f);
            s[j] = make_float2(0.f, 0.f);
            if (turned) {
                turn(pos, freq[lane * 4 + 2 * j], &c[j].x, &s[j].x);
                turn(pos, freq[lane * 4 + 2 * j + 1], &c[j].y, &s[j].y);
            }
        }
    }

    // x <- R x with (c, s), R^T x with (c, -s): its first four entries are the first ones
    // of the four pairs.  Entries that do not turn take c alone: a product with s = 0 would
    // hand on another entry's infinity as a NaN.
    __device__ __forceinline__ void rotate(float2 (&x)[4], const float2 (&c)[2], const float2 (&s)[2]) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 a = x[j], b = x[j + 2], minus = make_float2(-s[j].x, -s[j].y);
            x[j] = __fmul2_rn(a, c[j]);
            x[j + 2] = __fmul2_rn(b, c[j]);
            if (turned) {
                x[j] = __ffma2_rn(b, minus, x[j]);
                x[j + 2] = __ffma2_rn(a, s[j], x[j + 2]);
            }
        }
    }
};

// Forward: a group takes one item, its rows' loads kFwdRows at a time in registers.
template <typename T, int G, bool HALVES>
__global__ void __launch_bounds__(kThreads) qk_rotate_fwd_kernel(const __grid_constant__ QkParams p) {
    constexpr bool RUN = !HALVES, PAIRS = !HALVES;
    __shared__ uint2 freq[128];
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) freq[i] = p.freq[i];
    __syncthreads();
    // a CTA's groups take items of one side, or (both) a token's heads of q, then of k
    const int side = blockIdx.x >= p.side[0].ctas;
    const unsigned cta = side ? blockIdx.x - p.side[0].ctas : blockIdx.x;
    const int lane = threadIdx.x % G;
    const Lane<HALVES> l(lane, p.d, p.rot);
    const float inv_d = 1.f / (float)p.d;
    const Side& a = p.side[side];
    const Side& k = p.side[1];
    const int split = p.both ? a.H : a.hb, rows = split + (p.both ? k.H : 0);  // the same for every group
    const long long y_h = (long long)p.tokens.T * p.d;
    for (unsigned base = cta * (kThreads / G); base < a.items; base += a.ctas * (kThreads / G)) {
        const Place at(p, a, base + threadIdx.x / G);
        const int there = !l.on || at.heads == 0 ? 0 : p.both ? rows : at.heads;
        const T* a_row = (const T*)a.x + at.b * a.x_b + at.t * a.x_t + at.h0 * a.x_h;
        const T* k_row = (const T*)k.x + at.b * k.x_b + at.t * k.x_t;
        T* y_row = (T*)a.y + ((long long)at.b * a.H + at.h0) * y_h + (long long)at.t * p.d;
        Raw8<T> raw[kFwdRows];
        auto fetch = [&](int i) {
#pragma unroll
            for (int u = 0; u < kFwdRows; ++u) {
                raw[u].a = {};
                raw[u].b = {};
                const int h = i + u;
                if (h < there)
                    raw[u] = raw8<RUN>(h < split ? a_row + h * a.x_h : k_row + (h - split) * k.x_h, l.e1, l.e2);
            }
        };
        fetch(0);  // before the angles: their arithmetic covers the first loads
        float2 w[4], c[2], s[2];
        row_weights<PAIRS>(a.w, l.on, l.e1, l.e2, w);
        float scale = a.scale;
        l.angles(freq, lane,
                 p.positions ? __ldg(p.positions + (long long)at.b * p.tokens.T + at.t) : p.pos0 + at.t, c, s);
        for (int i = 0; i < rows; i += kFwdRows) {
            if (i > 0) fetch(i);
#pragma unroll
            for (int u = 0; u < kFwdRows; ++u) {
                const int h = i + u;
                if (h >= rows) break;
                if (h == split) {  // on to the keys
                    row_weights<PAIRS>(k.w, l.on, l.e1, l.e2, w);
                    scale = k.scale;
                    y_row = (T*)k.y + (long long)at.b * k.H * y_h + (long long)at.t * p.d;
                }
                float2 x[4];
                floats8<PAIRS>(raw[u], x);
                float f = scale;
                if (p.norm) f *= rsqrtf(group_sum<G>(dot8(x, x)) * inv_d + p.eps);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(x[j], __fmul2_rn(w[j], both(f)));
                l.rotate(x, c, s);
                if (h < there) store8<RUN, PAIRS>(y_row, l.e1, l.e2, x);
                y_row += y_h;
            }
        }
    }
}

// Backward: a CTA's groups walk items of one side; their rows come through the ring.
template <typename T, int G, bool HALVES>
__global__ void __launch_bounds__(kThreads, 5) qk_rotate_bwd_kernel(const __grid_constant__ QkParams p) {
    constexpr int kGroups = kThreads / G, kRing = kRingBytes / (int)sizeof(T), kSlot = 8 * G;
    constexpr bool RUN = !HALVES, PAIRS = !HALVES;
    __shared__ __align__(16) T ring[kRing][2][kGroups * kSlot];
    __shared__ uint2 freq[128];
    tc::griddep_launch_dependents();  // the sums' kernel may be scheduled (it waits itself)
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) freq[i] = p.freq[i];
    __syncthreads();
    const int key = blockIdx.x >= p.side[0].ctas;
    const Side& a = p.side[key];
    const unsigned cta = key ? blockIdx.x - p.side[0].ctas : blockIdx.x, leap = a.ctas * kGroups;
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const Lane<HALVES> l(lane, p.d, p.rot);
    const float inv_d = 1.f / (float)p.d;
    const long long g_h = (long long)p.tokens.T * p.d;

    // the fetching end: f_base is the CTA's first item (all groups take the same turns)
    unsigned f_base = cta * kGroups;
    int f_i = 0, f_heads = 0, f_slot = 0;
    const T *f_x = nullptr, *f_g = nullptr;
    auto fetch = [&]() {
        if (f_base < a.items) {
            if (f_i == 0) {
                const Place at(p, a, f_base + grp);
                f_heads = at.heads;
                f_x = (const T*)a.x + at.b * a.x_b + at.t * a.x_t + at.h0 * a.x_h;
                f_g = (const T*)a.g + (((long long)at.b * a.H + at.h0) * p.tokens.T + at.t) * p.d;
            }
            copy_row<T, G>(&ring[f_slot][0][grp * kSlot], f_x, lane, p.d, f_i < f_heads);
            copy_row<T, G>(&ring[f_slot][1][grp * kSlot], f_g, lane, p.d, f_i < f_heads);
            if (++f_i < f_heads) {
                f_x += a.x_h;
                f_g += g_h;
            }
            if (f_i == a.hb) {
                f_i = 0;
                f_base += leap;
            }
        }
        copies_commit();
        f_slot = f_slot + 1 == kRing ? 0 : f_slot + 1;
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch();

    float2 w[4], dw[4], c[2], s[2];
    row_weights<PAIRS>(a.w, l.on, l.e1, l.e2, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[j] = make_float2(0.f, 0.f);
    int slot = 0;
    auto position = [&](unsigned base) {
        const Place at(p, a, base + grp);
        return p.positions ? __ldg(p.positions + (long long)at.b * p.tokens.T + at.t) : p.pos0 + at.t;
    };
    int pos = position(cta * kGroups);
    for (unsigned base = cta * kGroups; base < a.items; base += leap) {
        const Place at(p, a, base + grp);
        const int heads = l.on ? at.heads : 0;
        l.angles(freq, lane, pos, c, s);
        if (base + leap < a.items) pos = position(base + leap);  // an item ahead
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // back, and the scale with it
            c[j] = __fmul2_rn(c[j], both(a.scale));
            s[j] = __fmul2_rn(s[j], both(-a.scale));
        }
        T* y = (T*)a.y + at.b * a.y_b + at.t * a.y_t + at.h0 * a.y_h;
        for (int i = 0; i < a.hb; ++i) {
            copies_wait<kRing - 1>();
            __syncwarp();
            float2 x[4], g[4];
            floats8<PAIRS>(raw8<RUN>(&ring[slot][0][grp * kSlot], l.e1, l.e2), x);
            floats8<PAIRS>(raw8<RUN>(&ring[slot][1][grp * kSlot], l.e1, l.e2), g);
            __syncwarp();
            fetch();
            slot = slot + 1 == kRing ? 0 : slot + 1;
            l.rotate(g, c, s);
            if (p.norm) {
                float2 gw[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) gw[j] = __fmul2_rn(g[j], w[j]);
                const float ss = group_sum<G>(dot8(x, x)), along = group_sum<G>(dot8(gw, x));
                const float n = rsqrtf(ss * inv_d + p.eps), back = -n * (n * along * inv_d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // rows that are not there hold zeros and add none
                    x[j] = __fmul2_rn(x[j], both(n));
                    dw[j] = __ffma2_rn(g[j], x[j], dw[j]);
                    g[j] = __ffma2_rn(x[j], both(back), __fmul2_rn(gw[j], both(n)));
                }
            }
            if (i < heads) store8<RUN, PAIRS>(y, l.e1, l.e2, g);
            y += a.y_h;
        }
    }
    if (!a.part) return;
    float* red = reinterpret_cast<float*>(&ring[0][0][0]);
    static_assert(sizeof(ring) >= kThreads * 8 * sizeof(float), "a thread's eight sums fit the ring");
    copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = entry8<PAIRS>(j >> 1, j & 1);
        if (l.on) red[grp * kSlot + (e < 4 ? l.e1 + e : l.e2 + e - 4)] = j & 1 ? dw[j >> 1].y : dw[j >> 1].x;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.d; e += kThreads) {
        float sum = 0.f;
        for (int i = 0; i < kGroups; ++i) sum += red[i * kSlot + e];
        a.part[(size_t)cta * p.d + e] = sum;
    }
}

constexpr int kFwdPerSm = 32, kBwdPerSm = 5;

// Heads a group walks: all of a side's (its angles are then computed once a token)
// while that leaves the card full of groups, fewer for short calls.
int head_block(const QkRotateArgs& a, int heads, int sms) {
    const long long threads = (long long)a.B * a.T * group_lanes(a.d), full = sms * 256LL;
    int hb = heads;
    while (hb > 1 && threads * ((heads + hb - 1) / hb) < full) hb = (hb + 1) / 2;
    return hb;
}

// One side's share of the groups and CTAs.  Backward, a few CTAs per SM stay and walk
// the items, each leaving one row of partial sums.
void plan_side(Side* s, const QkRotateArgs& a, bool key, bool bwd, int sms) {
    const int groups = kThreads / group_lanes(a.d);
    s->H = key ? a.Hk : a.Hq;
    s->hb = head_block(a, s->H, sms);
    s->nhb = (s->H + s->hb - 1) / s->hb;
    s->items = (unsigned)((long long)a.B * a.T * s->nhb);
    s->ctas = (s->items + groups - 1) / groups;
    // an item costs its heads' rows and, for its set-up and angles, about 1.5 rows more
    const double rows = s->hb + 1.5, share = s->nhb * rows;
    const int other = key ? a.Hq : a.Hk, other_hb = head_block(a, other, sms);
    const double rest = (double)((other + other_hb - 1) / other_hb) * (other_hb + 1.5);
    const double most = sms * (bwd ? kBwdPerSm : kFwdPerSm) * share / (share + rest);
    s->ctas = std::min(s->ctas, (unsigned)std::max(1.0, most));
}

// f / 2 pi modulo one turn in units of 2^-64 turns, |f| < 2^64: the product of f's 53 bits
// and 128 bits of 1 / 2 pi, each cut off: less than 2 units off.  In doubles it would be
// 2^-53 of f / 2 pi off: at a position of 2^31 that is 2^-22 radians for f = 1 and 2^-12
// for f = 1000.
unsigned long long turn_fraction(double f) {
    using Wide = unsigned __int128;
    constexpr unsigned long long kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // 2^128 / 2 pi
    int e;
    const auto m = (unsigned long long)std::ldexp(std::frexp(std::fabs(f), &e), 53);  // |f| = m 2^(e - 53)
    const Wide low = (Wide)m * kLo, high = (Wide)m * kHi + (low >> 64);  // m 2^128 / 2 pi = high 2^64 + low % 2^64
    const int s = 117 - e;  // its bits from 2^s on are the units, s >= 53
    unsigned long long F = 0;
    if (s < 64) F = (unsigned long long)(high << (64 - s)) | (unsigned long long)low >> s;
    else if (s < 192) F = (unsigned long long)(high >> (s - 64));
    return f < 0 ? 0ull - F : F;
}

QkParams params(const QkRotateArgs& a, bool bwd) {
    QkParams p;
    const int sms = sm_count();
    for (int key = 0; key < 2; ++key) {
        Side& s = p.side[key];
        const long long *xs = key ? a.k_strides : a.q_strides, *ys = key ? a.yk_strides : a.yq_strides;
        s.x = key ? a.k : a.q;
        s.g = key ? a.dk_out : a.dq_out;
        s.y = key ? a.yk : a.yq;
        s.w = key ? a.k_weight : a.q_weight;
        s.part = nullptr;
        s.x_b = xs[0]; s.x_t = xs[1]; s.x_h = xs[2];
        s.y_b = ys[0]; s.y_t = ys[1]; s.y_h = ys[2];
        s.scale = key ? a.k_scale : a.q_scale;
        plan_side(&s, a, key, bwd, sms);
    }
    // with few heads the angles are the larger part: one group then takes both sides
    p.both = !bwd && p.side[0].nhb == 1 && p.side[1].nhb == 1;
    if (p.both) {
        p.side[0].ctas += p.side[1].ctas;
        p.side[1].ctas = 0;
    }
    p.positions = a.positions; p.pos0 = a.pos0;
    p.tokens = Divide::by(a.T);
    p.d = a.d; p.rot = a.rot; p.norm = a.norm;
    p.eps = a.eps;
    for (int i = 0; i < a.rot / 2; ++i) {
        const unsigned long long F = turn_fraction(a.inv_freq[i]);
        p.freq[i] = make_uint2((unsigned)F, (unsigned)(F >> 32));
    }
    return p;
}

template <typename T, int G>
void launch(const QkParams& p, bool halves, bool bwd, unsigned grid, cudaStream_t s) {
    if (bwd) {
        if (halves) qk_rotate_bwd_kernel<T, G, true><<<grid, kThreads, 0, s>>>(p);
        else qk_rotate_bwd_kernel<T, G, false><<<grid, kThreads, 0, s>>>(p);
    } else {
        if (halves) qk_rotate_fwd_kernel<T, G, true><<<grid, kThreads, 0, s>>>(p);
        else qk_rotate_fwd_kernel<T, G, false><<<grid, kThreads, 0, s>>>(p);
    }
}

template <typename T>
void launch(const QkParams& p, bool halves, bool bwd, unsigned grid, cudaStream_t s) {
    switch (group_lanes(p.d)) {
        case 2: launch<T, 2>(p, halves, bwd, grid, s); break;
        case 4: launch<T, 4>(p, halves, bwd, grid, s); break;
        case 8: launch<T, 8>(p, halves, bwd, grid, s); break;
        case 16: launch<T, 16>(p, halves, bwd, grid, s); break;
        default: launch<T, 32>(p, halves, bwd, grid, s); break;
    }
}

}  // namespace

size_t qk_rotate_bwd_workspace_bytes(const QkRotateArgs& a) {
    Side q, k;
    const int sms = sm_count();
    plan_side(&q, a, false, true, sms);
    plan_side(&k, a, true, true, sms);
    return ((size_t)q.ctas + k.ctas) * a.d * sizeof(float);
}

cudaError_t launch_qk_rotate_fwd(const QkRotateArgs& a, cudaStream_t s) {
    const QkParams p = params(a, false);
    const unsigned grid = p.side[0].ctas + p.side[1].ctas;
    TraceScope trace("qk_rotate_fwd_kernel", s);
    if (a.bf16) launch<__nv_bfloat16>(p, a.halves, false, grid, s);
    else launch<float>(p, a.halves, false, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_qk_rotate_bwd(const QkRotateArgs& a, cudaStream_t s) {
    QkParams p = params(a, true);
    const unsigned grid = p.side[0].ctas + p.side[1].ctas;
    float* part = (float*)a.workspace;
    if (a.dq_weight) p.side[0].part = part;
    if (a.dk_weight) p.side[1].part = part + (size_t)p.side[0].ctas * a.d;
    {
        TraceScope trace("qk_rotate_bwd_kernel", s);
        if (a.bf16) launch<__nv_bfloat16>(p, a.halves, true, grid, s);
        else launch<float>(p, a.halves, true, grid, s);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(a.dq_weight || a.dk_weight)) return e;
    return launch_partial_sum(p.side[0].part, (int)p.side[0].ctas, a.dq_weight, p.side[1].part,
                              (int)p.side[1].ctas, a.dk_weight, a.d, s);
}

}  // namespace la
