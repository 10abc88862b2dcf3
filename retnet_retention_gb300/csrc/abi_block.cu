// The C ABI of the operators of a state space layer in its residual block
// (include/linattn.h: la_short_conv_*, la_ssm_*, la_block_norm_*): argument checks on
// the host, then asynchronous launches on the caller's stream.  Nothing is launched or
// written when a check fails.
#include <climits>
#include <cmath>
#include <cstring>

#include "abi_checks.h"
#include "launch.h"

using namespace la;

namespace {

// The view of a [B][T][D] tensor with two strides (batch, token) or null for dense.
bool make_rows(View* v, const void* p, const long long* strides, int B, int T, int D, la_dtype dtype) {
    const long long s[3] = {strides ? strides[0] : (long long)T * D, strides ? strides[1] : D, 0};
    return make_view(v, p, s, B, T, 1, D, dtype);
}

void keep(long long (&to)[2], const View& v) {
    to[0] = v.stride[0];
    to[1] = v.stride[1];
}

// Outputs as strided rows and as plain memory, inputs as memory: each output's rows apart,
// its memory apart from every input's and every other output's.
struct Memory {
    Region in[20];
    int n_in = 0;
    const View* out[8];
    int n_out = 0;
    Region flat[8];
    int n_flat = 0;

    void input(const void* p, size_t n) {
        if (p) in[n_in++] = {p, n};
    }
    void input(const View& v) { input(v.p, v.bytes()); }
    void output(const View& v) { out[n_out++] = &v; }
    void output(const void* p, size_t n) {
        if (p) flat[n_flat++] = {p, n};
    }
    bool ok() const {
        for (int i = 0; i < n_out; ++i) {
            if (!rows_apart(*out[i])) return false;
            for (int j = i + 1; j < n_out; ++j)
                if (overlap(*out[i], *out[j])) return false;
            for (int j = 0; j < n_flat; ++j)
                if (overlap(*out[i], flat[j].p, flat[j].n)) return false;
            for (int j = 0; j < n_in; ++j)
                if (overlap(*out[i], in[j].p, in[j].n)) return false;
        }
        for (int i = 0; i < n_flat; ++i) {
            for (int j = i + 1; j < n_flat; ++j)
                if (ranges_overlap(flat[i].p, flat[i].n, flat[j].p, flat[j].n)) return false;
            for (int j = 0; j < n_in; ++j)
                if (ranges_overlap(flat[i].p, flat[i].n, in[j].p, in[j].n)) return false;
        }
        return true;
    }
};

constexpr long long kMaxChannels = 1ll << 33;  // of all sequences together

constexpr long long kMaxTokens = (1ll << 31) - 256;  // a token a tile further still is an int

bool rows_shape_ok(int B, int T, int D, la_dtype dtype) {
    return B >= 0 && T >= 0 && D >= 16 && D % 16 == 0 && valid_dtype(dtype) && (long long)B * T <= kMaxTokens &&
           (B == 0 || T == 0 || (long long)B * T <= kMaxSpan / D) && (long long)B * D <= kMaxChannels;
}

// ---- short_conv ----------------------------------------------------------------------

bool conv_shape_ok(int B, int T, int D, int W, la_dtype dtype) {
    return rows_shape_ok(B, T, D, dtype) && W >= 2 && W <= 4 && (long long)D * W <= INT_MAX;
}

la_status conv_args(ShortConvArgs* a, const float* weight, const float* bias, la_dtype dtype, int B, int T,
                    int D, int W, unsigned flags) {
    if (!conv_shape_ok(B, T, D, W, dtype) || (flags & ~LA_CONV_SILU)) return LA_ERR_INVALID_ARG;
    std::memset(a, 0, sizeof(*a));
    a->B = B; a->T = T; a->D = D; a->W = W;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->silu = (flags & LA_CONV_SILU) != 0;
    a->weight = weight; a->bias = bias;
    if ((long long)B * T == 0) return LA_OK;
    if (!weight || any_misaligned({weight, bias})) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

// ---- ssm -----------------------------------------------------------------------------

bool ssm_shape_ok(int B, int T, int D, int N, int G, la_dtype dtype) {
    return rows_shape_ok(B, T, D, dtype) && B <= 65535 && (N == 8 || N == 16 || N == 32 || N == 64) && G >= 1 && G <= 65535 &&
           D % G == 0 && D / G % 8 == 0 && (long long)D * N <= INT_MAX && (long long)G * N <= INT_MAX &&
           (long long)B * D * N <= kMaxChannels;
}

// What the forward, the backward and the single-token call share.
la_status ssm_args(SsmArgs* a, const float* A, const float* skip, const float* dt_bias, la_dtype dtype, int B,
                   int T, int D, int N, int G, unsigned flags) {
    if (!ssm_shape_ok(B, T, D, N, G, dtype) || (flags & ~LA_SSM_SOFTPLUS)) return LA_ERR_INVALID_ARG;
    std::memset(a, 0, sizeof(*a));
    a->B = B; a->T = T; a->D = D; a->N = N; a->G = G;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->softplus = (flags & LA_SSM_SOFTPLUS) != 0;
    a->A = A; a->skip = skip; a->dt_bias = dt_bias;
    if ((long long)B * T == 0) return LA_OK;
    if (!A || any_misaligned({A, skip, dt_bias})) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

// The five inputs' views from pairs of strides; gate may be null.
bool ssm_views(SsmArgs* a, View (&v)[5], const void* x, const void* dt, const void* b, const void* c,
               const void* gate, const long long* strides, la_dtype dtype) {
    const void* p[5] = {x, dt, b, c, gate};
    const void** at[5] = {&a->x, &a->dt, &a->bm, &a->cm, &a->gate};
    long long(*to[5])[2] = {&a->x_strides, &a->dt_strides, &a->b_strides, &a->c_strides, &a->gate_strides};
    for (int i = 0; i < 5; ++i) {
        v[i].p = nullptr;
        if (i == 4 && !gate) break;
        const int width = i == 2 || i == 3 ? a->G * a->N : a->D;
        if (!make_rows(&v[i], p[i], strides ? strides + 2 * i : nullptr, a->B, a->T, width, dtype)) return false;
        *at[i] = p[i];
        keep(*to[i], v[i]);
    }
    return true;
}

void ssm_inputs(Memory* m, const SsmArgs& a, const View (&v)[5]) {
    for (const View& i : v)
        if (i.p) m->input(i);
    m->input(a.A, (size_t)a.D * a.N * 4);
    m->input(a.skip, (size_t)a.D * 4);
    m->input(a.dt_bias, (size_t)a.D * 4);
}

// ---- block_norm ----------------------------------------------------------------------

constexpr unsigned kBlockFlags = LA_BLOCK_POST_NORM | LA_BLOCK_PRE_NORM | LA_BLOCK_CENTER | LA_BLOCK_GATE_EACH;

bool block_shape_ok(int B, int T, int D, la_dtype dtype, la_dtype residual) {
    return rows_shape_ok(B, T, D, dtype) && D <= 8192 && valid_dtype(residual) &&
           (residual == LA_DTYPE_F32 || dtype == LA_DTYPE_BF16) && B <= 65535;
}

la_status block_args(BlockNormArgs* a, View* vo, const void* o, const long long* o_strides, la_dtype dtype,
                     la_dtype residual, const float* post_weight, const float* gate, const float* pre_weight,
                     int B, int T, int D, unsigned flags, float scale, float residual_scale, float eps) {
    if (!block_shape_ok(B, T, D, dtype, residual) || (flags & ~kBlockFlags)) return LA_ERR_INVALID_ARG;
    if (!(std::isfinite(eps) && eps > 0.f) || !std::isfinite(scale) || !std::isfinite(residual_scale))
        return LA_ERR_INVALID_ARG;
    std::memset(a, 0, sizeof(*a));
    a->B = B; a->T = T; a->D = D;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->residual_bf16 = residual == LA_DTYPE_BF16;
    a->post = (flags & LA_BLOCK_POST_NORM) != 0;
    a->pre = (flags & LA_BLOCK_PRE_NORM) != 0;
    a->center = (flags & LA_BLOCK_CENTER) != 0;
    a->gate_each = (flags & LA_BLOCK_GATE_EACH) != 0;
    a->scale = scale; a->residual_scale = residual_scale; a->eps = eps;
    a->post_weight = post_weight; a->gate = gate; a->pre_weight = pre_weight;
    if ((post_weight && !a->post) || (pre_weight && !a->pre) || (a->gate_each && !gate)) return LA_ERR_INVALID_ARG;
    if ((long long)B * T == 0) return LA_OK;
    if (any_misaligned({post_weight, gate, pre_weight})) return LA_ERR_INVALID_ARG;
    if (!make_rows(vo, o, o_strides, B, T, D, dtype)) return LA_ERR_INVALID_ARG;
    a->o = o;
    keep(a->o_strides, *vo);
    return LA_OK;
}

size_t gate_bytes(const BlockNormArgs& a) { return (size_t)(a.gate_each ? a.B : 1) * a.D * 4; }

}  // namespace

extern "C" {

la_status la_short_conv_fwd(const void* x, const long long* x_strides, la_dtype dtype, const float* weight,
                            const float* bias, int B, int T, int D, int W, unsigned flags, const void* state,
                            const int* positions, void* y, const long long* y_strides, void* state_out,
                            la_stream_t stream) {
    ShortConvArgs a;
    const la_status st = conv_args(&a, weight, bias, dtype, B, T, D, W, flags);
    if (st != LA_OK) return st;
    if (any_misaligned({state, positions, state_out})) return LA_ERR_INVALID_ARG;
    if (B == 0) return LA_OK;
    const size_t es = elem_size(dtype), held = (size_t)B * (W - 1) * D * es;
    cudaStream_t s = (cudaStream_t)stream;
    if (state != state_out && ranges_overlap(state, held, state_out, held)) return LA_ERR_INVALID_ARG;
    if (T == 0) {  // no token: the state stays as it is (its bytes, as fp32 words)
        if (!state_out) return LA_OK;
        return cuda_status(state ? launch_state_copy((float*)state_out, (const float*)state, held / 4, s)
                                 : launch_state_zero((float*)state_out, nullptr, held / 4, 0, s));
    }
    View vx, vy;
    if (!make_rows(&vx, x, x_strides, B, T, D, dtype) || !make_rows(&vy, y, y_strides, B, T, D, dtype))
        return LA_ERR_INVALID_ARG;
    Memory m;
    m.input(vx);
    m.input(weight, (size_t)D * W * 4);
    m.input(bias, (size_t)D * 4);
    m.input(positions, (size_t)B * T * 4);
    if (state != state_out) m.input(state, held);
    m.output(vy);
    m.output(state_out, held);
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.x = x; a.y = y; a.state = state; a.state_out = state_out; a.positions = positions;
    keep(a.x_strides, vx);
    keep(a.y_strides, vy);
    return cuda_status(launch_short_conv_fwd(a, s));
}

size_t la_short_conv_bwd_workspace_size(int B, int T, int D, int W, la_dtype dtype) {
    if (!conv_shape_ok(B, T, D, W, dtype) || (long long)B * T == 0) return 0;
    ShortConvArgs a;
    std::memset(&a, 0, sizeof(a));
    a.B = B; a.T = T; a.D = D; a.W = W;
    a.bf16 = dtype == LA_DTYPE_BF16;
    return short_conv_bwd_workspace_bytes(a);
}

la_status la_short_conv_bwd(const void* x, const long long* x_strides, const void* dy,
                            const long long* dy_strides, la_dtype dtype, const float* weight,
                            const float* bias, int B, int T, int D, int W, unsigned flags, const void* state,
                            const int* positions, const void* dstate_T, void* dx, const long long* dx_strides,
                            float* dweight, float* dbias, void* dstate, void* workspace,
                            size_t workspace_bytes, la_stream_t stream) {
    ShortConvArgs a;
    const la_status st = conv_args(&a, weight, bias, dtype, B, T, D, W, flags);
    if (st != LA_OK) return st;
    if (any_misaligned({state, positions, dstate_T, dweight, dbias, dstate, workspace})) return LA_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype), held = (size_t)B * (W - 1) * D * es;
    const size_t wb = (size_t)D * W * 4, bb = (size_t)D * 4;
    cudaStream_t s = (cudaStream_t)stream;
    Memory m;
    m.input(dstate_T, held);
    m.output(dweight, wb);
    m.output(dbias, bb);
    m.output(dstate, held);
    if ((long long)B * T == 0) {  // the sums over no tokens; the state's gradient passes through
        if (!m.ok()) return LA_ERR_INVALID_ARG;
        cudaError_t e = cudaSuccess;
        if (dweight) e = launch_state_zero(dweight, nullptr, (size_t)D * W, 0, s);
        if (dbias && e == cudaSuccess) e = launch_state_zero(dbias, nullptr, D, 0, s);
        if (dstate && B > 0 && e == cudaSuccess)
            e = dstate_T ? launch_state_copy((float*)dstate, (const float*)dstate_T, held / 4, s)
                         : launch_state_zero((float*)dstate, nullptr, held / 4, 0, s);
        return cuda_status(e);
    }
    const size_t need = dweight || dbias ? short_conv_bwd_workspace_bytes(a) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return LA_ERR_INVALID_ARG;
    View vx, vdy, vdx;
    if (!make_rows(&vx, x, x_strides, B, T, D, dtype) || !make_rows(&vdy, dy, dy_strides, B, T, D, dtype) ||
        !make_rows(&vdx, dx, dx_strides, B, T, D, dtype))
        return LA_ERR_INVALID_ARG;
    m.input(vx);
    m.input(vdy);
    m.input(weight, wb);
    m.input(bias, bb);
    m.input(positions, (size_t)B * T * 4);
    m.input(state, held);
    m.output(vdx);
    m.output(need ? workspace : nullptr, need);
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.x = x; a.dy = dy; a.dx = dx;
    a.state = state; a.positions = positions; a.dstate_T = dstate_T; a.dstate = dstate;
    a.dweight = dweight; a.dbias = dbias;
    a.workspace = workspace;
    keep(a.x_strides, vx);
    keep(a.dy_strides, vdy);
    keep(a.dx_strides, vdx);
    return cuda_status(launch_short_conv_bwd(a, s));
}

la_status la_short_conv_step_at(const void* x, long long x_stride, la_dtype dtype, const float* weight,
                                const float* bias, int B, int D, int W, unsigned flags, const void* state,
                                const int* positions, void* state_out, void* y, la_stream_t stream) {
    ShortConvArgs a;
    const la_status st = conv_args(&a, weight, bias, dtype, B, 1, D, W, flags);
    if (st != LA_OK || B == 0) return st;
    if (!state || !state_out || !y || any_misaligned({state, positions, state_out, y})) return LA_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype), held = (size_t)B * (W - 1) * D * es;
    const long long xs[2] = {x_stride, 0};
    View vx;
    if (!make_rows(&vx, x, xs, B, 1, D, dtype)) return LA_ERR_INVALID_ARG;
    if (state != state_out && ranges_overlap(state, held, state_out, held)) return LA_ERR_INVALID_ARG;
    Memory m;
    m.input(vx);
    m.input(weight, (size_t)D * W * 4);
    m.input(bias, (size_t)D * 4);
    m.input(positions, (size_t)B * 4);
    if (state != state_out) m.input(state, held);
    m.output(state_out, held);
    m.output(y, (size_t)B * D * es);
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.x = x; a.y = y; a.state = state; a.state_out = state_out; a.positions = positions;
    keep(a.x_strides, vx);
    return cuda_status(launch_short_conv_step(a, (cudaStream_t)stream));
}

la_status la_short_conv_step(const void* x, long long x_stride, la_dtype dtype, const float* weight,
                             const float* bias, int B, int D, int W, unsigned flags, const void* state,
                             void* state_out, void* y, la_stream_t stream) {
    return la_short_conv_step_at(x, x_stride, dtype, weight, bias, B, D, W, flags, state, nullptr, state_out, y,
                                 stream);
}

la_status la_ssm_fwd(const void* x, const void* dt, const float* A, const void* b, const void* c,
                     const float* skip, const void* gate, const float* dt_bias, const long long* strides,
                     la_dtype dtype, int B, int T, int D, int N, int G, unsigned flags, const float* h0,
                     const int* positions, void* y, float* h_out, void* workspace, size_t workspace_bytes,
                     la_stream_t stream) {
    SsmArgs a;
    const la_status st = ssm_args(&a, A, skip, dt_bias, dtype, B, T, D, N, G, flags);
    if (st != LA_OK) return st;
    if (any_misaligned({h0, positions, h_out, workspace})) return LA_ERR_INVALID_ARG;
    if (B == 0) return LA_OK;
    const size_t state = (size_t)B * D * N;
    cudaStream_t s = (cudaStream_t)stream;
    if (h0 != h_out && ranges_overlap(h0, state * 4, h_out, state * 4)) return LA_ERR_INVALID_ARG;
    if (T == 0) {  // no token: the final state is the initial one
        if (!h_out) return LA_OK;
        return cuda_status(h0 ? launch_state_copy(h_out, h0, state, s)
                              : launch_state_zero(h_out, nullptr, state, 0, s));
    }
    const size_t need = ssm_workspace_bytes(a);
    if (workspace_bytes < need || (need > 0 && !workspace)) return LA_ERR_INVALID_ARG;
    View in[5], vy;
    if (!ssm_views(&a, in, x, dt, b, c, gate, strides, dtype) ||
        !make_rows(&vy, y, strides ? strides + 10 : nullptr, B, T, D, dtype))
        return LA_ERR_INVALID_ARG;
    Memory m;
    ssm_inputs(&m, a, in);
    m.input(positions, (size_t)B * T * 4);
    if (h0 != h_out) m.input(h0, state * 4);
    m.output(vy);
    m.output(h_out, state * 4);
    m.output(need ? workspace : nullptr, need);
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.positions = positions; a.h0 = h0; a.h_out = h_out; a.y = y;
    a.workspace = workspace;
    keep(a.y_strides, vy);
    return cuda_status(launch_ssm_fwd(a, s));
}

size_t la_ssm_workspace_size(int B, int T, int D, int N, int G, la_dtype dtype) {
    SsmArgs a;
    if (ssm_args(&a, nullptr, nullptr, nullptr, dtype, B, 0, D, N, G, 0) != LA_OK ||
        !ssm_shape_ok(B, T, D, N, G, dtype) || (long long)B * T == 0)
        return 0;
    a.T = T;
    return ssm_workspace_bytes(a);
}

size_t la_ssm_bwd_workspace_size(int B, int T, int D, int N, int G, la_dtype dtype) {
    SsmArgs a;
    if (ssm_args(&a, nullptr, nullptr, nullptr, dtype, B, 0, D, N, G, 0) != LA_OK ||
        !ssm_shape_ok(B, T, D, N, G, dtype) || (long long)B * T == 0)
        return 0;
    a.T = T;
    return ssm_bwd_workspace_bytes(a);
}

la_status la_ssm_bwd(const void* x, const void* dt, const float* A, const void* b, const void* c,
                     const float* skip, const void* gate, const float* dt_bias, const void* dy,
                     const long long* strides, la_dtype dtype, int B, int T, int D, int N, int G,
                     unsigned flags, const float* h0, const int* positions, const float* dh_T, void* dx,
                     void* ddt, float* dA, void* db, void* dc, float* dskip, void* dgate, float* ddt_bias,
                     float* dh0, void* workspace, size_t workspace_bytes, la_stream_t stream) {
    SsmArgs a;
    const la_status st = ssm_args(&a, A, skip, dt_bias, dtype, B, T, D, N, G, flags);
    if (st != LA_OK) return st;
    if (any_misaligned({h0, positions, dh_T, dA, dskip, ddt_bias, dh0, workspace})) return LA_ERR_INVALID_ARG;
    const size_t state = (size_t)B * D * N, wa = (size_t)D * N * 4, wd = (size_t)D * 4;
    cudaStream_t s = (cudaStream_t)stream;
    Memory m;
    m.input(dh_T, state * 4);
    m.output(dA, wa);
    m.output(dskip, wd);
    m.output(ddt_bias, wd);
    m.output(dh0, state * 4);
    if ((long long)B * T == 0) {  // the sums over no tokens; the state's gradient passes through
        if (!m.ok()) return LA_ERR_INVALID_ARG;
        cudaError_t e = cudaSuccess;
        if (dA) e = launch_state_zero(dA, nullptr, (size_t)D * N, 0, s);
        if (dskip && e == cudaSuccess) e = launch_state_zero(dskip, nullptr, D, 0, s);
        if (ddt_bias && e == cudaSuccess) e = launch_state_zero(ddt_bias, nullptr, D, 0, s);
        if (dh0 && B > 0 && e == cudaSuccess)
            e = dh_T ? launch_state_copy(dh0, dh_T, state, s) : launch_state_zero(dh0, nullptr, state, 0, s);
        return cuda_status(e);
    }
    if ((gate == nullptr) != (dgate == nullptr)) return LA_ERR_INVALID_ARG;
    const size_t need = ssm_bwd_workspace_bytes(a);
    if (workspace_bytes < need || !workspace) return LA_ERR_INVALID_ARG;
    View in[5], vdy, out[5];
    if (!ssm_views(&a, in, x, dt, b, c, gate, strides, dtype) ||
        !make_rows(&vdy, dy, strides ? strides + 10 : nullptr, B, T, D, dtype))
        return LA_ERR_INVALID_ARG;
    void* p[5] = {dx, ddt, db, dc, dgate};
    long long(*to[5])[2] = {&a.dx_strides, &a.ddt_strides, &a.db_strides, &a.dc_strides, &a.dgate_strides};
    for (int i = 0; i < (gate ? 5 : 4); ++i) {
        const int width = i == 2 || i == 3 ? G * N : D;
        if (!make_rows(&out[i], p[i], strides ? strides + 12 + 2 * i : nullptr, B, T, width, dtype))
            return LA_ERR_INVALID_ARG;
        keep(*to[i], out[i]);
        m.output(out[i]);
    }
    ssm_inputs(&m, a, in);
    m.input(vdy);
    m.input(positions, (size_t)B * T * 4);
    m.input(h0, state * 4);
    m.output(workspace, need);
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.dy = dy;
    keep(a.dy_strides, vdy);
    a.positions = positions; a.h0 = h0; a.dh_T = dh_T;
    a.dx = dx; a.ddt = ddt; a.db = db; a.dc = dc; a.dgate = dgate;
    a.dA = dA; a.dskip = dskip; a.ddt_bias = ddt_bias; a.dh0 = dh0;
    a.workspace = workspace;
    return cuda_status(launch_ssm_bwd(a, s));
}

la_status la_ssm_step(const void* x, const void* dt, const float* A, const void* b, const void* c,
                      const float* skip, const void* gate, const float* dt_bias, const long long* strides,
                      la_dtype dtype, int B, int D, int N, int G, unsigned flags, const float* h_in,
                      float* h_out, void* y, la_stream_t stream) {
    SsmArgs a;
    const la_status st = ssm_args(&a, A, skip, dt_bias, dtype, B, 1, D, N, G, flags);
    if (st != LA_OK || B == 0) return st;
    if (!h_in || !h_out || !y || any_misaligned({h_in, h_out, y})) return LA_ERR_INVALID_ARG;
    long long pairs[10] = {0};
    for (int i = 0; strides && i < 5; ++i) pairs[2 * i] = strides[i];
    View in[5];
    if (!ssm_views(&a, in, x, dt, b, c, gate, strides ? pairs : nullptr, dtype)) return LA_ERR_INVALID_ARG;
    const size_t state = (size_t)B * D * N * 4;
    if (h_in != h_out && ranges_overlap(h_in, state, h_out, state)) return LA_ERR_INVALID_ARG;
    Memory m;
    ssm_inputs(&m, a, in);
    if (h_in != h_out) m.input(h_in, state);
    m.output(h_out, state);
    m.output(y, (size_t)B * D * elem_size(dtype));
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.h0 = h_in; a.h_out = h_out; a.y = y;
    return cuda_status(launch_ssm_step(a, (cudaStream_t)stream));
}

la_status la_block_norm_fwd(const void* o, const long long* o_strides, la_dtype dtype, const void* h,
                            const long long* h_strides, la_dtype residual_dtype, const float* post_weight,
                            const float* gate, const float* pre_weight, int B, int T, int D, unsigned flags,
                            float scale, float residual_scale, float eps, void* h_out,
                            const long long* h_out_strides, void* y, const long long* y_strides,
                            la_stream_t stream) {
    BlockNormArgs a;
    View vo, vh, vho, vy;
    const la_status st = block_args(&a, &vo, o, o_strides, dtype, residual_dtype, post_weight, gate, pre_weight,
                                    B, T, D, flags, scale, residual_scale, eps);
    if (st != LA_OK || (long long)B * T == 0) return st;
    if (a.pre != (y != nullptr) || (!h_out && !y)) return LA_ERR_INVALID_ARG;
    if ((h && !make_rows(&vh, h, h_strides, B, T, D, residual_dtype)) ||
        (h_out && !make_rows(&vho, h_out, h_out_strides, B, T, D, residual_dtype)) ||
        (y && !make_rows(&vy, y, y_strides, B, T, D, dtype)))
        return LA_ERR_INVALID_ARG;
    Memory m;
    m.input(vo);
    // in place: a row is read whole before it is written
    const bool in_place = h && h == h_out && vh.stride[0] == vho.stride[0] && vh.stride[1] == vho.stride[1];
    if (h && !in_place) m.input(vh);
    m.input(post_weight, (size_t)D * 4);
    m.input(gate, gate_bytes(a));
    m.input(pre_weight, (size_t)D * 4);
    if (h_out) m.output(vho);
    if (y) m.output(vy);
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.h = h; a.h_out = h_out; a.y = y;
    if (h) keep(a.h_strides, vh);
    if (h_out) keep(a.h_out_strides, vho);
    if (y) keep(a.y_strides, vy);
    return cuda_status(launch_block_norm_fwd(a, (cudaStream_t)stream));
}

size_t la_block_norm_bwd_workspace_size(int B, int T, int D, la_dtype dtype, unsigned flags) {
    if (!block_shape_ok(B, T, D, dtype, LA_DTYPE_F32) || (flags & ~kBlockFlags) || (long long)B * T == 0) return 0;
    BlockNormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.B = B; a.T = T; a.D = D;
    a.bf16 = dtype == LA_DTYPE_BF16;
    a.gate_each = (flags & LA_BLOCK_GATE_EACH) != 0;
    static const float present = 1.f;
    a.gate = a.gate_each ? &present : nullptr;  // only whether there is one counts
    return block_norm_bwd_workspace_bytes(a);
}

la_status la_block_norm_bwd(const void* o, const long long* o_strides, la_dtype dtype, const void* h_out,
                            const long long* h_out_strides, la_dtype residual_dtype, const void* dy,
                            const long long* dy_strides, const void* dh_out, const long long* dh_out_strides,
                            const float* post_weight, const float* gate, const float* pre_weight, int B, int T,
                            int D, unsigned flags, float scale, float residual_scale, float eps, void* d_o,
                            const long long* d_o_strides, void* dh, const long long* dh_strides,
                            float* dpost_weight, float* dgate, float* dpre_weight, void* workspace,
                            size_t workspace_bytes, la_stream_t stream) {
    BlockNormArgs a;
    View vo, vh, vdy, vdh, vdo, vdr;
    const la_status st = block_args(&a, &vo, o, o_strides, dtype, residual_dtype, post_weight, gate, pre_weight,
                                    B, T, D, flags, scale, residual_scale, eps);
    if (st != LA_OK) return st;
    if ((dpost_weight && !post_weight) || (dgate && !gate) || (dpre_weight && !pre_weight) ||
        any_misaligned({dpost_weight, dgate, dpre_weight, workspace}))
        return LA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t wb = (size_t)D * 4;
    Memory m;
    m.output(dpost_weight, wb);
    m.output(dgate, gate_bytes(a));
    m.output(dpre_weight, wb);
    if ((long long)B * T == 0) {  // the sums over no tokens
        if (!m.ok()) return LA_ERR_INVALID_ARG;
        cudaError_t e = cudaSuccess;
        if (dpost_weight) e = launch_state_zero(dpost_weight, nullptr, D, 0, s);
        if (dgate && gate_bytes(a) > 0 && e == cudaSuccess)
            e = launch_state_zero(dgate, nullptr, gate_bytes(a) / 4, 0, s);
        if (dpre_weight && e == cudaSuccess) e = launch_state_zero(dpre_weight, nullptr, D, 0, s);
        return cuda_status(e);
    }
    if (a.pre != (dy != nullptr) || (a.pre && !h_out) || (!dy && !dh_out)) return LA_ERR_INVALID_ARG;
    const size_t need = dpost_weight || dgate || dpre_weight ? block_norm_bwd_workspace_bytes(a) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return LA_ERR_INVALID_ARG;
    if ((a.pre && !make_rows(&vh, h_out, h_out_strides, B, T, D, residual_dtype)) ||
        (dy && !make_rows(&vdy, dy, dy_strides, B, T, D, dtype)) ||
        (dh_out && !make_rows(&vdh, dh_out, dh_out_strides, B, T, D, residual_dtype)) ||
        !make_rows(&vdo, d_o, d_o_strides, B, T, D, dtype) ||
        (dh && !make_rows(&vdr, dh, dh_strides, B, T, D, residual_dtype)))
        return LA_ERR_INVALID_ARG;
    m.input(vo);
    if (a.pre) m.input(vh);
    if (dy) m.input(vdy);
    const bool in_place = dh && dh == dh_out && vdr.stride[0] == vdh.stride[0] && vdr.stride[1] == vdh.stride[1];
    if (dh_out && !in_place) m.input(vdh);
    m.input(post_weight, wb);
    m.input(gate, gate_bytes(a));
    m.input(pre_weight, wb);
    m.output(vdo);
    if (dh) m.output(vdr);
    m.output(need ? workspace : nullptr, need);
    if (!m.ok()) return LA_ERR_INVALID_ARG;
    a.h = a.pre ? h_out : nullptr; a.dy = dy; a.dh = dh_out; a.d_o = d_o; a.d_res = dh;
    if (a.pre) keep(a.h_strides, vh);
    if (dy) keep(a.dy_strides, vdy);
    if (dh_out) keep(a.dh_strides, vdh);
    keep(a.d_o_strides, vdo);
    if (dh) keep(a.d_res_strides, vdr);
    a.dpost_weight = dpost_weight; a.dgate = dgate; a.dpre_weight = dpre_weight;
    a.workspace = workspace;
    return cuda_status(launch_block_norm_bwd(a, s));
}

}  // extern "C"
