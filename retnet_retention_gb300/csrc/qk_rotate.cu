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
// integers: F_i = f_i / 2 pi in units of 2^-64 turns, p F_i mod 2^64 is exact, so a
// position of any size keeps the angle to fp32 accuracy, without 64-bit floats.
//
// Bound by HBM: 2 bytes in and 2 out an entry (bf16), about 10 operations.  A
// group of d / 8 lanes holds one row.  With split halves a lane holds four entries
// of the first half and the four they pair with, so that the rotation needs no
// exchange between lanes.  A group keeps its token and walks heads: the four angles
// of a lane are computed once for a block of heads.
#include <algorithm>
#include <cmath>

#include "rows.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;  // rows (heads) whose loads are in flight together

struct QkParams {
    const void *q, *k;            // raw projections
    const void *gq, *gk;          // backward: gradients of the outputs [B][H][T][d]
    void *yq, *yk;                // outputs, or the projections' gradients
    const float *wq, *wk;         // norm weights [d] or null
    float* part;                  // backward: per-CTA weight gradients [CTA][2][d] or null
    long long q_sb, q_st, q_sh, k_sb, k_st, k_sh;      // elements
    long long yq_sb, yq_st, yq_sh, yk_sb, yk_st, yk_sh;
    const int* positions;         // [B][T] or null: pos0 + t
    int pos0, B, T, Hq, Hk, d, rot, norm;
    int hb, nhb;                  // heads a group walks, blocks of heads
    unsigned items;               // B nhb T: what the groups share out
    float eps, q_scale, k_scale;
    unsigned long long freq[128]; // turns per position, units of 2^-64

    // Neighbouring groups take neighbouring tokens: their output rows touch.
    __device__ __forceinline__ void place(unsigned item, int* t, int* hblk, int* b) const {
        const unsigned row = item / (unsigned)T;
        *t = (int)(item - row * (unsigned)T);
        *b = (int)(row / (unsigned)nhb);
        *hblk = (int)(row - (unsigned)*b * (unsigned)nhb);
    }
};

// cos and sin of p F turns: the nearest quarter turn apart, the rest (at most an
// eighth of a turn) to fp32.
__device__ __forceinline__ void turn(unsigned long long frac, float* c, float* s) {
    const unsigned quarter = (unsigned)((frac + (1ull << 61)) >> 62);
    const int rest = (int)((frac - ((unsigned long long)quarter << 62)) >> 32);
    float s0, c0;
    sincospif((float)rest * 4.656612873077393e-10f, &s0, &c0);  // 2^-31: half turns
    const float cc = (quarter & 1) ? s0 : c0, ss = (quarter & 1) ? c0 : s0;
    *c = ((quarter + 1) & 2) ? -cc : cc;
    *s = (quarter & 2) ? -ss : ss;
}

// A lane's entries and angles: entries e1..e1+3 and e2..e2+3; in the rotated part
// its four pairs are number 4 lane + j, (j, j + 4) of its eight with split halves
// and (2j, 2j + 1) with adjacent ones.
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

    __device__ __forceinline__ void angles(const unsigned long long* freq, int lane, int pos,
                                           float (&c)[4], float (&s)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = 1.f;
            s[j] = 0.f;
            if (turned) turn((unsigned long long)(long long)pos * freq[lane * 4 + j], &c[j], &s[j]);
        }
    }

    // x <- R x (dir = 1) or R^T x (dir = -1)
    __device__ __forceinline__ static void rotate(float (&x)[8], const float (&c)[4],
                                                  const float (&s)[4], float dir) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i1 = HALVES ? j : 2 * j, i2 = HALVES ? j + 4 : 2 * j + 1;
            const float a = x[i1], b = x[i2], sj = dir * s[j];
            x[i1] = a * c[j] - b * sj;
            x[i2] = a * sj + b * c[j];
        }
    }
};

template <bool HALVES>
__device__ __forceinline__ void load_weights(const float* w, const Lane<HALVES>& l, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 1.f;
    if (w && l.on) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = __ldg(w + l.e1 + j);
            x[j + 4] = __ldg(w + l.e2 + j);
        }
    }
}

template <typename T, int G, bool HALVES>
__global__ void __launch_bounds__(kThreads) qk_rotate_fwd_kernel(const __grid_constant__ QkParams p) {
    __shared__ unsigned long long freq[128];
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) freq[i] = p.freq[i];
    __syncthreads();
    const int lane = threadIdx.x % G;
    const unsigned item = blockIdx.x * (kThreads / G) + threadIdx.x / G;
    const bool live = item < p.items;  // whole groups; dead ones keep the shuffles company
    int t, hblk, b;
    p.place(live ? item : 0, &t, &hblk, &b);
    const Lane<HALVES> l(lane, p.d, p.rot);
    const int pos = p.positions ? __ldg(p.positions + (long long)b * p.T + t) : p.pos0 + t;
    float c[4], s[4];
    l.angles(freq, lane, pos, c, s);
    float wq[8], wk[8];
    load_weights<HALVES>(p.wq, l, wq);
    load_weights<HALVES>(p.wk, l, wk);
    const T* q = (const T*)p.q + b * p.q_sb + t * p.q_st;
    const T* k = (const T*)p.k + b * p.k_sb + t * p.k_st;
    const float inv_d = 1.f / (float)p.d;
    const int heads = p.Hq + p.Hk;
    for (int i = 0; i < p.hb; i += kRows) {
        const int h0 = hblk * p.hb + i;
        Raw8<T> raw[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = h0 + u;
            const T* row = h < p.Hq ? q + h * p.q_sh : k + (h - p.Hq) * p.k_sh;
            raw[u] = live && l.on && i + u < p.hb && h < heads ? load_raw8<!HALVES>(row, l.e1, l.e2)
                                                               : zero_raw8<T>();
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (i + u >= p.hb) break;  // the same for every group
            const int h = h0 + u;
            const bool key = h >= p.Hq;
            float x[8];
            floats8(raw[u], x);
            float f = key ? p.k_scale : p.q_scale;
            if (p.norm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
                f *= rsqrtf(group_sum<G>(ss) * inv_d + p.eps);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= f * (key ? wk[j] : wq[j]);
            Lane<HALVES>::rotate(x, c, s, 1.f);
            if (live && l.on && h < heads) {
                T* y = key ? (T*)p.yk + (((long long)b * p.Hk + (h - p.Hq)) * p.T + t) * p.d
                           : (T*)p.yq + (((long long)b * p.Hq + h) * p.T + t) * p.d;
                store8<!HALVES>(y, l.e1, l.e2, x);
            }
        }
    }
}

template <typename T, int G, bool HALVES>
__global__ void __launch_bounds__(kThreads) qk_rotate_bwd_kernel(const __grid_constant__ QkParams p) {
    __shared__ unsigned long long freq[128];
    __shared__ float red[(kThreads / G) * G * 8];
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) freq[i] = p.freq[i];
    __syncthreads();
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    constexpr int kGroups = kThreads / G;
    const Lane<HALVES> l(lane, p.d, p.rot);
    float wq[8], wk[8], dwq[8], dwk[8];
    load_weights<HALVES>(p.wq, l, wq);
    load_weights<HALVES>(p.wk, l, wk);
#pragma unroll
    for (int j = 0; j < 8; ++j) dwq[j] = dwk[j] = 0.f;
    const float inv_d = 1.f / (float)p.d;
    // the bound is the CTA's first item: every group of a warp takes the same turns
    for (unsigned base = blockIdx.x * kGroups; base < p.items; base += gridDim.x * kGroups) {
        const unsigned item = base + grp;
        const bool live = item < p.items;
        int t, hblk, b;
        p.place(live ? item : 0, &t, &hblk, &b);
        const int pos = p.positions ? __ldg(p.positions + (long long)b * p.T + t) : p.pos0 + t;
        float c[4], s[4];
        l.angles(freq, lane, pos, c, s);
        for (int i = 0; i < p.hb; ++i) {  // the same for every group, dead ones too
            const int h = hblk * p.hb + i;
            const bool key = h >= p.Hq, row_on = live && l.on && h < p.Hq + p.Hk;
            const int hh = key ? h - p.Hq : h;
            Raw8<T> rx = zero_raw8<T>(), rg = zero_raw8<T>();
            if (row_on) {
                const T* xr = key ? (const T*)p.k + b * p.k_sb + t * p.k_st + hh * p.k_sh
                                  : (const T*)p.q + b * p.q_sb + t * p.q_st + hh * p.q_sh;
                const T* gr = key ? (const T*)p.gk + (((long long)b * p.Hk + hh) * p.T + t) * p.d
                                  : (const T*)p.gq + (((long long)b * p.Hq + hh) * p.T + t) * p.d;
                rx = load_raw8<!HALVES>(xr, l.e1, l.e2);
                rg = load_raw8<!HALVES>(gr, l.e1, l.e2);
            }
            float x[8], g[8];
            floats8(rx, x);
            floats8(rg, g);
            const float scale = key ? p.k_scale : p.q_scale;
            Lane<HALVES>::rotate(g, c, s, -1.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] *= scale;
            if (p.norm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
                const float r = rsqrtf(group_sum<G>(ss) * inv_d + p.eps);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] *= r;
                    if (row_on) {
                        if (key) dwk[j] += g[j] * x[j];
                        else dwq[j] += g[j] * x[j];
                    }
                    g[j] *= key ? wk[j] : wq[j];
                    dot += g[j] * x[j];
                }
                dot = group_sum<G>(dot) * inv_d;
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = r * (g[j] - x[j] * dot);
            }
            if (row_on) {
                T* y = key ? (T*)p.yk + b * p.yk_sb + t * p.yk_st + hh * p.yk_sh
                           : (T*)p.yq + b * p.yq_sb + t * p.yq_st + hh * p.yq_sh;
                store8<!HALVES>(y, l.e1, l.e2, g);
            }
        }
    }
    if (!p.part) return;
#pragma unroll 1
    for (int m = 0; m < 2; ++m) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (l.on) red[grp * G * 8 + (j < 4 ? l.e1 + j : l.e2 + j - 4)] = m ? dwk[j] : dwq[j];
        __syncthreads();
        for (int e = threadIdx.x; e < p.d; e += kThreads) {
            float sum = 0.f;
            for (int i = 0; i < kGroups; ++i) sum += red[i * G * 8 + e];
            p.part[((size_t)blockIdx.x * 2 + m) * p.d + e] = sum;
        }
    }
}

// Heads a group walks: all of them (its angles are then computed once a token)
// while that leaves the card full of groups, fewer for short calls.
int head_block(const QkRotateArgs& a) {
    const long long threads = (long long)a.B * a.T * group_lanes(a.d), full = sm_count() * 1024LL;
    const int heads = a.Hq + a.Hk;
    int hb = heads;
    while (hb > 1 && threads * ((heads + hb - 1) / hb) < full) hb = (hb + 1) / 2;
    return hb;
}

// CTAs of the backward kernel: a few per SM, each leaving one row of partial sums.
int bwd_ctas(const QkRotateArgs& a) {
    const int groups = kThreads / group_lanes(a.d), hb = head_block(a);
    const long long items = (long long)a.B * a.T * ((a.Hq + a.Hk + hb - 1) / hb);
    return (int)std::min<long long>((items + groups - 1) / groups, sm_count() * 4LL);
}

QkParams params(const QkRotateArgs& a) {
    QkParams p;
    p.q = a.q; p.k = a.k; p.gq = a.dq_out; p.gk = a.dk_out;
    p.yq = a.yq; p.yk = a.yk;
    p.wq = a.q_weight; p.wk = a.k_weight;
    p.part = nullptr;
    p.q_sb = a.q_strides[0]; p.q_st = a.q_strides[1]; p.q_sh = a.q_strides[2];
    p.k_sb = a.k_strides[0]; p.k_st = a.k_strides[1]; p.k_sh = a.k_strides[2];
    p.yq_sb = a.yq_strides[0]; p.yq_st = a.yq_strides[1]; p.yq_sh = a.yq_strides[2];
    p.yk_sb = a.yk_strides[0]; p.yk_st = a.yk_strides[1]; p.yk_sh = a.yk_strides[2];
    p.positions = a.positions; p.pos0 = a.pos0;
    p.B = a.B; p.T = a.T; p.Hq = a.Hq; p.Hk = a.Hk; p.d = a.d; p.rot = a.rot; p.norm = a.norm;
    p.eps = a.eps; p.q_scale = a.q_scale; p.k_scale = a.k_scale;
    p.hb = head_block(a);
    p.nhb = (a.Hq + a.Hk + p.hb - 1) / p.hb;
    p.items = (unsigned)((long long)a.B * a.T * p.nhb);
    for (int i = 0; i < 128; ++i) p.freq[i] = 0;
    for (int i = 0; i < a.rot / 2; ++i) {
        // the fraction of a turn per position, in [0, 1): whole turns change nothing
        double turns = a.inv_freq[i] * 0.15915494309189533577;
        turns -= std::floor(turns);
        p.freq[i] = turns >= 1.0 ? 0ull : (unsigned long long)std::ldexp(turns, 64);
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
    return (size_t)bwd_ctas(a) * 2 * a.d * sizeof(float);
}

cudaError_t launch_qk_rotate_fwd(const QkRotateArgs& a, cudaStream_t s) {
    const QkParams p = params(a);
    const unsigned groups = kThreads / group_lanes(a.d), grid = (p.items + groups - 1) / groups;
    TraceScope trace("qk_rotate_fwd_kernel", s);
    if (a.bf16) launch<__nv_bfloat16>(p, a.halves, false, grid, s);
    else launch<float>(p, a.halves, false, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_qk_rotate_bwd(const QkRotateArgs& a, cudaStream_t s) {
    QkParams p = params(a);
    const int grid = bwd_ctas(a);
    const bool sums = a.dq_weight || a.dk_weight;
    p.part = sums ? (float*)a.workspace : nullptr;
    {
        TraceScope trace("qk_rotate_bwd_kernel", s);
        if (a.bf16) launch<__nv_bfloat16>(p, a.halves, true, (unsigned)grid, s);
        else launch<float>(p, a.halves, true, (unsigned)grid, s);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !sums) return e;
    return launch_partial_sum(p.part, grid, a.dq_weight, a.d, a.dk_weight, a.d, s);
}

}  // namespace la
