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
// Bound by HBM: o and h in, h' and y out.  A CTA holds a row in registers (a thread eight
// neighbouring entries, once or twice), so that both norms cost no second read; the
// next row's loads are in flight meanwhile.  y is the norm of h' before its rounding; the
// gradients start from the rounded h' that the forward call left.
#include <algorithm>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

struct Rows {
    const void* p;
    long long b, t;  // strides
};

struct BlockParams {
    Rows o, h, dy, dh;             // h: the residual, backward h'; null pointers where absent
    Rows h_out, y, d_o, d_res;     // outputs
    const float *w_post, *gate, *w_pre;
    float *part_post, *part_gate, *part_pre;  // backward: partial rows, or null
    int B, T, D;
    int rows_cta;                  // rows a CTA holds at once
    int seq_blocks;                // CTAs a sequence's rows are shared out to (0: of all sequences)
    int post, pre, center, gate_each;
    float alpha, beta, eps;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float2 (&x)[4]) {
    floats8<false>(raw8<true>(p, 0, 4), x);
}

// Sums of N values over the threads of a row, in a fixed order.  `red`: 2 x [warps][N] a
// row in turn, so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& turn, int warps, int warp) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<32>(v[i]);
    if (warps == 1) return;
    float* to = red + turn * 16 * 2;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) to[warp * 2 + i] = v[i];
    }
    __syncthreads();
    float s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
    for (int k = 0; k < warps; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += to[k * 2 + i];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = s[i];
}

__device__ __forceinline__ float sum8(const float2 (&x)[4]) {
    const float2 s = __fadd2_rn(__fadd2_rn(x[0], x[1]), __fadd2_rn(x[2], x[3]));
    return s.x + s.y;
}

// A thread's place: row slot, its warp in the row, its first entry.
struct Place {
    int slot, warp, warps, lane;
    __device__ Place(int rows_cta) {
        const int per = blockDim.x / rows_cta;
        slot = threadIdx.x / per;
        lane = threadIdx.x - slot * per;
        warps = per / 32;
        warp = lane / 32;
    }
};

// T: o and y; R: the residual stream.  P pieces of eight entries a thread.
template <typename T, typename R, int P>
__global__ void __launch_bounds__(512) block_norm_kernel(const __grid_constant__ BlockParams p) {
    __shared__ float red[4][2 * 16 * 2];
    const Place at(p.rows_cta);
    const int width = at.warps * 32 * 8;  // entries of a piece of the row
    const long long rows = (long long)p.B * p.T, leap = (long long)gridDim.x * p.rows_cta;
    const float inv_d = 1.f / (float)p.D;
    int turn = 0;
    bool on[P];
    int e[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        e[i] = i * width + at.lane * 8;
        on[i] = e[i] < p.D;
    }
    Raw8<T> o_next[P];
    Raw8<R> h_next[P];
    auto fetch = [&](long long m) {
        if (m >= rows) return;
        const long long b = m / p.T, t = m - b * p.T;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (on[i]) {
                o_next[i] = raw8<true>((const T*)p.o.p + b * p.o.b + t * p.o.t + e[i], 0, 4);
                if (p.h.p) h_next[i] = raw8<true>((const R*)p.h.p + b * p.h.b + t * p.h.t + e[i], 0, 4);
            }
    };
    long long m = (long long)blockIdx.x * p.rows_cta + at.slot;
    fetch(m);
    for (; m - at.slot < rows; m += leap) {  // the same for every slot
        const bool row = m < rows;
        const long long b = row ? m / p.T : 0, t = row ? m - b * p.T : 0;
        float2 v[P][4], h[P][4];
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = h[i][j] = make_float2(0.f, 0.f);
        if (row) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (on[i]) {
                    floats8<false>(o_next[i], v[i]);
                    if (p.h.p) floats8<false>(h_next[i], h[i]);
                }
        }
        fetch(m + leap);
        auto normed = [&](float2 (&x)[P][4]) {
            if (p.center) {
                float s[1] = {0.f};
#pragma unroll
                for (int i = 0; i < P; ++i) s[0] += sum8(x[i]);
                row_sums<1>(s, red[at.slot], turn, at.warps, at.warp);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (on[i])
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[i][j] = __fadd2_rn(x[i][j], both(-s[0] * inv_d));
            }
            float q[1] = {0.f};
#pragma unroll
            for (int i = 0; i < P; ++i) q[0] += dot8(x[i], x[i]);
            row_sums<1>(q, red[at.slot], turn, at.warps, at.warp);
            const float r = rsqrtf(q[0] * inv_d + p.eps);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = __fmul2_rn(x[i][j], both(r));
        };
        if (p.post) normed(v);
        const float* gate = p.gate ? p.gate + (p.gate_each ? b * p.D : 0) : nullptr;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 w[4], g[4];
            row_weights<false>(p.w_post, on[i], e[i], e[i] + 4, w);
            row_weights<false>(gate, on[i], e[i], e[i] + 4, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = __fmul2_rn(__fmul2_rn(v[i][j], w[j]), __fmul2_rn(g[j], both(p.alpha)));
                v[i][j] = __ffma2_rn(h[i][j], both(p.beta), v[i][j]);
            }
            if (row && on[i] && p.h_out.p)
                store8<true, false>((R*)p.h_out.p + b * p.h_out.b + t * p.h_out.t + e[i], 0, 4, v[i]);
        }
        if (!p.pre) continue;
        normed(v);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 w[4];
            row_weights<false>(p.w_pre, on[i], e[i], e[i] + 4, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], w[j]);
            if (row && on[i]) store8<true, false>((T*)p.y.p + b * p.y.b + t * p.y.t + e[i], 0, 4, v[i]);
        }
    }
}

// A CTA takes rows of one sequence where each sequence has its own gate (its sums then
// belong to that sequence's gradient), else of all.
template <typename T, typename R, int P>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const __grid_constant__ BlockParams p) {
    tc::griddep_launch_dependents();  // the sums' kernel may be scheduled (it waits itself)
    __shared__ float red[4][2 * 16 * 2];
    extern __shared__ float columns[];  // [rows_cta][D] for the sums over a CTA's row slots
    const Place at(p.rows_cta);
    const int width = at.warps * 32 * 8;
    const long long first_row = p.seq_blocks ? (long long)(blockIdx.x / p.seq_blocks) * p.T : 0;
    const long long end_row = p.seq_blocks ? first_row + p.T : (long long)p.B * p.T;
    const long long block = p.seq_blocks ? blockIdx.x % p.seq_blocks : blockIdx.x;
    const long long leap = (long long)(p.seq_blocks ? p.seq_blocks : gridDim.x) * p.rows_cta;
    const float inv_d = 1.f / (float)p.D;
    int turn = 0;
    bool on[P];
    int e[P];
    float2 s_post[P][4], s_gate[P][4], s_pre[P][4];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        e[i] = i * width + at.lane * 8;
        on[i] = e[i] < p.D;
#pragma unroll
        for (int j = 0; j < 4; ++j) s_post[i][j] = s_gate[i][j] = s_pre[i][j] = make_float2(0.f, 0.f);
    }
    for (long long m = first_row + block * p.rows_cta + at.slot; m - at.slot < end_row; m += leap) {
        const bool row = m < end_row;
        const long long b = row ? m / p.T : 0, t = row ? m - b * p.T : 0;
        float2 n[P][4], q[P][4], d[P][4], dt[P][4];  // norm(h'), p, dy, dt
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) n[i][j] = q[i][j] = d[i][j] = dt[i][j] = make_float2(0.f, 0.f);
            if (row && on[i]) {
                load8((const T*)p.o.p + b * p.o.b + t * p.o.t + e[i], q[i]);
                if (p.pre) {
                    load8((const R*)p.h.p + b * p.h.b + t * p.h.t + e[i], n[i]);
                    load8((const T*)p.dy.p + b * p.dy.b + t * p.dy.t + e[i], d[i]);
                }
                if (p.dh.p) load8((const R*)p.dh.p + b * p.dh.b + t * p.dh.t + e[i], dt[i]);
            }
        }
        // both rows' norms: means, then squares
        if (p.center) {
            float s[2] = {0.f, 0.f};
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
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) s[0] += dot8(n[i], n[i]), s[1] += dot8(q[i], q[i]);
        row_sums<2>(s, red[at.slot], turn, at.warps, at.warp);
        const float rh = rsqrtf(s[0] * inv_d + p.eps), ro = p.post ? rsqrtf(s[1] * inv_d + p.eps) : 1.f;
        if (p.pre) {
            s[0] = s[1] = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 w[4];
                row_weights<false>(p.w_pre, on[i], e[i], e[i] + 4, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[i][j] = __fmul2_rn(n[i][j], both(rh));
                    s_pre[i][j] = __ffma2_rn(d[i][j], n[i][j], s_pre[i][j]);
                    d[i][j] = __fmul2_rn(d[i][j], w[j]);
                }
                s[0] += dot8(d[i], n[i]);
                s[1] += sum8(d[i]);
            }
            row_sums<2>(s, red[at.slot], turn, at.warps, at.warp);
            const float2 along = both(-s[0] * inv_d), mean = both(p.center ? -s[1] * inv_d : 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (on[i])
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dt[i][j] = __ffma2_rn(both(rh), __ffma2_rn(n[i][j], along, __fadd2_rn(d[i][j], mean)),
                                              dt[i][j]);
        }
        const float* gate = p.gate ? p.gate + (p.gate_each ? b * p.D : 0) : nullptr;
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (row && on[i] && p.d_res.p) {
                float2 out[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) out[j] = __fmul2_rn(dt[i][j], both(p.beta));
                store8<true, false>((R*)p.d_res.p + b * p.d_res.b + t * p.d_res.t + e[i], 0, 4, out);
            }
            float2 w[4], g[4];
            row_weights<false>(p.w_post, on[i], e[i], e[i] + 4, w);
            row_weights<false>(gate, on[i], e[i], e[i] + 4, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[i][j] = __fmul2_rn(q[i][j], both(ro));
                dt[i][j] = __fmul2_rn(dt[i][j], both(p.alpha));
                s_gate[i][j] = __ffma2_rn(dt[i][j], __fmul2_rn(q[i][j], w[j]), s_gate[i][j]);
                dt[i][j] = __fmul2_rn(dt[i][j], g[j]);
                s_post[i][j] = __ffma2_rn(dt[i][j], q[i][j], s_post[i][j]);
                dt[i][j] = __fmul2_rn(dt[i][j], w[j]);
            }
            s[0] += dot8(dt[i], q[i]);
            s[1] += sum8(dt[i]);
        }
        if (p.post) {
            row_sums<2>(s, red[at.slot], turn, at.warps, at.warp);
            const float2 along = both(-s[0] * inv_d), mean = both(p.center ? -s[1] * inv_d : 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dt[i][j] = __fmul2_rn(both(ro), __ffma2_rn(q[i][j], along, __fadd2_rn(dt[i][j], mean)));
        }
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (row && on[i]) store8<true, false>((T*)p.d_o.p + b * p.d_o.b + t * p.d_o.t + e[i], 0, 4, dt[i]);
    }
    // one partial row a CTA, over its row slots
    auto leave = [&](const float2 (&sum)[P][4], float* part) {
        if (!part) return;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (on[i])
                store8<true, false>(columns + (size_t)at.slot * p.D + e[i], 0, 4, sum[i]);
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            float v = 0.f;
            for (int k = 0; k < p.rows_cta; ++k) v += columns[(size_t)k * p.D + c];
            part[(size_t)blockIdx.x * p.D + c] = v;
        }
    };
    leave(s_post, p.part_post);
    leave(s_gate, p.part_gate);
    leave(s_pre, p.part_pre);
}

// d(gate) of each sequence: its CTAs' partial rows, added in order.
__global__ void __launch_bounds__(128) block_gate_sum_kernel(const float* part, int blocks, int D, float* out) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    tc::griddep_wait();
    if (c >= D) return;
    const float* from = part + (size_t)blockIdx.y * blocks * D + c;
    float v = 0.f;
    for (int k = 0; k < blocks; ++k) v += from[(size_t)k * D];
    out[(size_t)blockIdx.y * D + c] = v;
}

struct Shape {
    int pieces, threads, rows;  // a row's pieces a thread and threads, rows a CTA
};

Shape shape(int D) {
    Shape s;
    s.pieces = D <= 4096 ? 1 : 2;
    const int per = 8 * s.pieces;
    s.threads = ((D + per - 1) / per + 31) / 32 * 32;
    s.rows = s.threads <= 32 ? 4 : s.threads <= 64 ? 2 : 1;
    return s;
}

constexpr int kFwdThreadsPerSm = 2048, kBwdThreadsPerSm = 1024;

long long fwd_blocks(const BlockNormArgs& a) {
    const Shape sh = shape(a.D);
    const long long rows = ((long long)a.B * a.T + sh.rows - 1) / sh.rows;
    return std::min(rows, (long long)sm_count() * (kFwdThreadsPerSm / (sh.threads * sh.rows)));
}

// CTAs of the gradients: (of each sequence, in all).
void bwd_blocks(const BlockNormArgs& a, int* each, long long* all) {
    const Shape sh = shape(a.D);
    const long long most = (long long)sm_count() * std::max(1, kBwdThreadsPerSm / (sh.threads * sh.rows));
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
    auto rows = [](const void* p, const long long* s) { return Rows{p, s[0], s[1]}; };
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
    p.post = a.post; p.pre = a.pre; p.center = a.center; p.gate_each = a.gate_each;
    p.alpha = a.scale; p.beta = a.residual_scale; p.eps = a.eps;
    return p;
}

template <typename T, typename R, int P>
cudaError_t launch(const BlockParams& p, bool bwd, unsigned grid, int threads, size_t shared, cudaStream_t s) {
    if (!bwd) {
        block_norm_kernel<T, R, P><<<grid, threads, 0, s>>>(p);
        return cudaGetLastError();
    }
    const cudaError_t e = cudaFuncSetAttribute(block_norm_bwd_kernel<T, R, P>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e != cudaSuccess) return e;
    block_norm_bwd_kernel<T, R, P><<<grid, threads, shared, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t launch(const BlockParams& p, bool bwd, unsigned grid, size_t shared, cudaStream_t s) {
    const Shape sh = shape(p.D);
    const int threads = sh.threads * sh.rows;
    return sh.pieces == 1 ? launch<T, R, 1>(p, bwd, grid, threads, shared, s)
                          : launch<T, R, 2>(p, bwd, grid, threads, shared, s);
}

cudaError_t launch(const BlockNormArgs& a, const BlockParams& p, bool bwd, unsigned grid, size_t shared,
                   cudaStream_t s) {
    if (!a.bf16) return launch<float, float>(p, bwd, grid, shared, s);
    if (a.residual_bf16) return launch<__nv_bfloat16, __nv_bfloat16>(p, bwd, grid, shared, s);
    return launch<__nv_bfloat16, float>(p, bwd, grid, shared, s);
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
    return launch(a, params(a), false, (unsigned)fwd_blocks(a), 0, s);
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, cudaStream_t s) {
    BlockParams p = params(a);
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
        e = launch(a, p, true, (unsigned)all, sums ? (size_t)p.rows_cta * a.D * sizeof(float) : 0, s);
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
