// The C ABI of the operators around retention (include/linattn.h: la_qk_rotate_*,
// la_head_gate_*, la_scan_*): argument checks on the host, then asynchronous
// launches on the caller's stream.  Nothing is launched or written when a check
// fails.
#include <climits>
#include <cmath>
#include <cstring>

#include "abi_checks.h"
#include "launch.h"

using namespace la;

namespace {

// ---- qk_rotate -----------------------------------------------------------------------

constexpr unsigned kQkFlags = LA_QK_NORM | LA_QK_ADJACENT;

bool qk_shape_ok(int B, int T, int Hq, int Hk, int d, la_dtype dtype) {
    return B >= 0 && T >= 0 && Hq >= 1 && Hk >= 1 && Hq <= 65536 && Hk <= 65536 && valid_width(d) &&
           valid_dtype(dtype) && (long long)B * T <= INT_MAX;
}

// Everything the forward and the backward call share; fills a and the views.
la_status qk_args(QkRotateArgs* a, View* vq, View* vk, const void* q, const long long* q_strides,
                  const void* k, const long long* k_strides, la_dtype dtype, int B, int T, int Hq,
                  int Hk, int d, int rot, const double* inv_freq, const int* positions, int pos0,
                  const float* q_weight, const float* k_weight, float eps, float q_scale,
                  float k_scale, unsigned flags) {
    if (!qk_shape_ok(B, T, Hq, Hk, d, dtype)) return LA_ERR_INVALID_ARG;
    if (rot < 0 || rot > d || rot % 16 != 0 || (flags & ~kQkFlags)) return LA_ERR_INVALID_ARG;
    const bool norm = (flags & LA_QK_NORM) != 0;
    if (norm && !(std::isfinite(eps) && eps > 0.f)) return LA_ERR_INVALID_ARG;
    if (!norm && (q_weight || k_weight)) return LA_ERR_INVALID_ARG;
    if (!std::isfinite(q_scale) || !std::isfinite(k_scale)) return LA_ERR_INVALID_ARG;
    if (rot > 0) {
        if (!inv_freq) return LA_ERR_INVALID_ARG;
        for (int i = 0; i < rot / 2; ++i)
            if (!(std::fabs(inv_freq[i]) < 18446744073709551616.0)) return LA_ERR_INVALID_ARG;  // or NaN
    }
    std::memset(a, 0, sizeof(*a));
    a->B = B; a->T = T; a->Hq = Hq; a->Hk = Hk; a->d = d; a->rot = rot;
    a->inv_freq = inv_freq; a->positions = positions; a->pos0 = pos0;
    a->q_weight = q_weight; a->k_weight = k_weight;
    a->eps = eps; a->q_scale = q_scale; a->k_scale = k_scale;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->norm = norm;
    a->halves = rot > 0 && !(flags & LA_QK_ADJACENT);
    a->q = q; a->k = k;
    if ((long long)B * T == 0) return LA_OK;
    if (!positions && (pos0 < 0 || (long long)pos0 + T - 1 > INT_MAX)) return LA_ERR_INVALID_ARG;
    if (!make_view(vq, q, q_strides, B, T, Hq, d, dtype) || !make_view(vk, k, k_strides, B, T, Hk, d, dtype))
        return LA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)positions, (const void*)q_weight, (const void*)k_weight})
        if (p && !aligned16(p)) return LA_ERR_INVALID_ARG;
    keep(a->q_strides, *vq);
    keep(a->k_strides, *vk);
    return LA_OK;
}

// ---- head_gate -----------------------------------------------------------------------

bool gate_shape_ok(int B, int H, int T, int d, la_dtype dtype) {
    return B >= 0 && T >= 0 && H >= 1 && H <= 65536 && valid_width(d) && valid_dtype(dtype) &&
           (long long)B * T <= INT_MAX;
}

la_status gate_args(HeadGateArgs* a, View* vo, View* vg, const void* o, const long long* o_strides,
                    const void* gate, const long long* gate_strides, la_dtype dtype,
                    const float* weight, int B, int H, int T, int d, unsigned flags, float eps) {
    if (!gate_shape_ok(B, H, T, d, dtype) || (flags & ~LA_GATE_CENTER)) return LA_ERR_INVALID_ARG;
    if (!(std::isfinite(eps) && eps > 0.f)) return LA_ERR_INVALID_ARG;
    std::memset(a, 0, sizeof(*a));
    a->B = B; a->H = H; a->T = T; a->d = d;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->center = (flags & LA_GATE_CENTER) != 0;
    a->eps = eps;
    a->o = o; a->gate = gate; a->weight = weight;
    if ((long long)B * T == 0) return LA_OK;
    if (!make_view(vo, o, o_strides, B, H, T, d, dtype)) return LA_ERR_INVALID_ARG;
    if (gate && !make_view(vg, gate, gate_strides, B, T, H, d, dtype)) return LA_ERR_INVALID_ARG;
    if (weight && !aligned16(weight)) return LA_ERR_INVALID_ARG;
    keep(a->o_strides, *vo);
    if (gate) keep(a->gate_strides, *vg);
    return LA_OK;
}

// ---- scan ----------------------------------------------------------------------------

// Channels of all sequences together.  They are at most 2^29 tiles of 32 (sequences of 16
// channels fill half a tile each), and so many tiles are one CTA each: a grid's limit is
// 2^31 - 1.
constexpr long long kMaxChannels = 1ll << 33;

bool scan_shape_ok(int B, int T, int D, la_dtype dtype) {
    return B >= 0 && T >= 0 && D >= 16 && D % 16 == 0 && valid_dtype(dtype) &&
           (B == 0 || T == 0 || (long long)B * T <= kMaxSpan / D) && (long long)B * D <= kMaxChannels;
}

}  // namespace

extern "C" {

la_status la_qk_rotate_fwd(const void* q, const long long* q_strides, const void* k,
                           const long long* k_strides, la_dtype dtype, int B, int T, int Hq, int Hk,
                           int d, int rot, const double* inv_freq, const int* positions, int pos0,
                           const float* q_weight, const float* k_weight, float eps, float q_scale,
                           float k_scale, unsigned flags, void* q_out, void* k_out,
                           la_stream_t stream) {
    QkRotateArgs a;
    View vq, vk;
    const la_status st = qk_args(&a, &vq, &vk, q, q_strides, k, k_strides, dtype, B, T, Hq, Hk, d,
                                 rot, inv_freq, positions, pos0, q_weight, k_weight, eps, q_scale,
                                 k_scale, flags);
    if (st != LA_OK) return st;
    const size_t tokens = (size_t)B * T, row = (size_t)d * elem_size(dtype);
    if (tokens == 0) return LA_OK;
    if (!q_out || !k_out || !aligned16(q_out) || !aligned16(k_out)) return LA_ERR_INVALID_ARG;
    const Region oq = {q_out, tokens * Hq * row}, ok = {k_out, tokens * Hk * row};
    if (clash({{q, vq.bytes()}, {k, vk.bytes()}, {positions, tokens * 4}, {q_weight, (size_t)d * 4},
               {k_weight, (size_t)d * 4}},
              {oq, ok}))
        return LA_ERR_INVALID_ARG;
    a.yq = q_out;
    a.yk = k_out;
    return cuda_status(launch_qk_rotate_fwd(a, (cudaStream_t)stream));
}

size_t la_qk_rotate_bwd_workspace_size(int B, int T, int Hq, int Hk, int d, la_dtype dtype) {
    if (!qk_shape_ok(B, T, Hq, Hk, d, dtype) || (long long)B * T == 0) return 0;
    QkRotateArgs a;
    std::memset(&a, 0, sizeof(a));
    a.B = B; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d;
    a.bf16 = dtype == LA_DTYPE_BF16;
    return qk_rotate_bwd_workspace_bytes(a);
}

la_status la_qk_rotate_bwd(const void* q, const long long* q_strides, const void* k,
                           const long long* k_strides, const void* dq_out, const void* dk_out,
                           la_dtype dtype, int B, int T, int Hq, int Hk, int d, int rot,
                           const double* inv_freq, const int* positions, int pos0,
                           const float* q_weight, const float* k_weight, float eps, float q_scale,
                           float k_scale, unsigned flags, void* dq, const long long* dq_strides,
                           void* dk, const long long* dk_strides, float* dq_weight,
                           float* dk_weight, void* workspace, size_t workspace_bytes,
                           la_stream_t stream) {
    QkRotateArgs a;
    View vq, vk, wq, wk;
    const la_status st = qk_args(&a, &vq, &vk, q, q_strides, k, k_strides, dtype, B, T, Hq, Hk, d,
                                 rot, inv_freq, positions, pos0, q_weight, k_weight, eps, q_scale,
                                 k_scale, flags);
    if (st != LA_OK) return st;
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return LA_ERR_INVALID_ARG;
    if (any_misaligned({dq_weight, dk_weight, workspace})) return LA_ERR_INVALID_ARG;
    const size_t tokens = (size_t)B * T, row = (size_t)d * elem_size(dtype), wb = (size_t)d * 4;
    cudaStream_t s = (cudaStream_t)stream;
    if (ranges_overlap(dq_weight, wb, dk_weight, wb)) return LA_ERR_INVALID_ARG;
    if (tokens == 0) {  // the sum over no tokens
        cudaError_t e = cudaSuccess;
        if (dq_weight) e = launch_state_zero(dq_weight, nullptr, d, 0, s);
        if (dk_weight && e == cudaSuccess) e = launch_state_zero(dk_weight, nullptr, d, 0, s);
        return cuda_status(e);
    }
    const size_t need = dq_weight || dk_weight ? qk_rotate_bwd_workspace_bytes(a) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return LA_ERR_INVALID_ARG;
    if (!dq_out || !dk_out || !aligned16(dq_out) || !aligned16(dk_out)) return LA_ERR_INVALID_ARG;
    if (!make_view(&wq, dq, dq_strides, B, T, Hq, d, dtype) ||
        !make_view(&wk, dk, dk_strides, B, T, Hk, d, dtype) || !rows_apart(wq) || !rows_apart(wk) ||
        overlap(wq, wk))
        return LA_ERR_INVALID_ARG;
    const Region ins[] = {{q, vq.bytes()}, {k, vk.bytes()}, {dq_out, tokens * Hq * row},
                          {dk_out, tokens * Hk * row}, {positions, tokens * 4}, {q_weight, wb},
                          {k_weight, wb}};
    const Region flat[] = {{dq_weight, wb}, {dk_weight, wb}, {workspace, need}};
    for (const Region& i : ins) {
        if (overlap(wq, i.p, i.n) || overlap(wk, i.p, i.n)) return LA_ERR_INVALID_ARG;
        for (const Region& o : flat)
            if (ranges_overlap(o.p, o.n, i.p, i.n)) return LA_ERR_INVALID_ARG;
    }
    for (const Region& o : flat)
        if (overlap(wq, o.p, o.n) || overlap(wk, o.p, o.n)) return LA_ERR_INVALID_ARG;
    if (ranges_overlap(dq_weight, wb, workspace, need) || ranges_overlap(dk_weight, wb, workspace, need))
        return LA_ERR_INVALID_ARG;
    a.dq_out = dq_out;
    a.dk_out = dk_out;
    a.yq = dq;
    a.yk = dk;
    keep(a.yq_strides, wq);
    keep(a.yk_strides, wk);
    a.dq_weight = dq_weight;
    a.dk_weight = dk_weight;
    a.workspace = workspace;
    return cuda_status(launch_qk_rotate_bwd(a, s));
}

la_status la_head_gate_fwd(const void* o, const long long* o_strides, const void* gate,
                           const long long* gate_strides, la_dtype dtype, const float* weight, int B,
                           int H, int T, int d, unsigned flags, float eps, void* y,
                           const long long* y_strides, la_stream_t stream) {
    HeadGateArgs a;
    View vo, vg, vy;
    const la_status st = gate_args(&a, &vo, &vg, o, o_strides, gate, gate_strides, dtype, weight, B,
                                   H, T, d, flags, eps);
    if (st != LA_OK || (long long)B * T == 0) return st;
    if (!make_view(&vy, y, y_strides, B, T, H, d, dtype) || !rows_apart(vy)) return LA_ERR_INVALID_ARG;
    if (overlap(vy, o, vo.bytes()) || (gate && overlap(vy, gate, vg.bytes())) ||
        overlap(vy, weight, (size_t)H * d * 4))
        return LA_ERR_INVALID_ARG;
    a.y = y;
    keep(a.y_strides, vy);
    return cuda_status(launch_head_gate_fwd(a, (cudaStream_t)stream));
}

size_t la_head_gate_bwd_workspace_size(int B, int H, int T, int d, la_dtype dtype) {
    if (!gate_shape_ok(B, H, T, d, dtype) || (long long)B * T == 0) return 0;
    HeadGateArgs a;
    std::memset(&a, 0, sizeof(a));
    a.B = B; a.H = H; a.T = T; a.d = d;
    a.bf16 = dtype == LA_DTYPE_BF16;
    return head_gate_bwd_workspace_bytes(a);
}

la_status la_head_gate_bwd(const void* o, const long long* o_strides, const void* gate,
                           const long long* gate_strides, const void* dy,
                           const long long* dy_strides, la_dtype dtype, const float* weight, int B,
                           int H, int T, int d, unsigned flags, float eps, void* d_o,
                           const long long* do_strides, void* dgate, const long long* dgate_strides,
                           float* dweight, void* workspace, size_t workspace_bytes,
                           la_stream_t stream) {
    HeadGateArgs a;
    View vo, vg, vdy, wo, wg;
    const la_status st = gate_args(&a, &vo, &vg, o, o_strides, gate, gate_strides, dtype, weight, B,
                                   H, T, d, flags, eps);
    if (st != LA_OK) return st;
    if (dweight && !weight) return LA_ERR_INVALID_ARG;
    if (any_misaligned({dweight, workspace})) return LA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t wb = (size_t)H * d * 4;
    if ((long long)B * T == 0)
        return dweight ? cuda_status(launch_state_zero(dweight, nullptr, (size_t)H * d, 0, s)) : LA_OK;
    if ((gate == nullptr) != (dgate == nullptr)) return LA_ERR_INVALID_ARG;
    const size_t need = dweight ? head_gate_bwd_workspace_bytes(a) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return LA_ERR_INVALID_ARG;
    if (!make_view(&vdy, dy, dy_strides, B, T, H, d, dtype) ||
        !make_view(&wo, d_o, do_strides, B, H, T, d, dtype) || !rows_apart(wo) ||
        (gate && (!make_view(&wg, dgate, dgate_strides, B, T, H, d, dtype) || !rows_apart(wg))))
        return LA_ERR_INVALID_ARG;
    const Region ins[] = {{o, vo.bytes()}, {gate, gate ? vg.bytes() : 0}, {dy, vdy.bytes()}, {weight, wb}};
    const Region outs[] = {{d_o, wo.bytes()}, {dgate, gate ? wg.bytes() : 0}, {dweight, wb}, {workspace, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Region& in : ins)
            if (ranges_overlap(outs[i].p, outs[i].n, in.p, in.n)) return LA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (ranges_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return LA_ERR_INVALID_ARG;
    }
    a.dy = dy;
    a.d_o = d_o;
    a.d_gate = dgate;
    keep(a.dy_strides, vdy);
    keep(a.do_strides, wo);
    if (gate) keep(a.dgate_strides, wg);
    a.d_weight = dweight;
    a.workspace = workspace;
    return cuda_status(launch_head_gate_bwd(a, s));
}

la_status la_scan_fwd(const void* x, la_dtype dtype, const float* log_a, int B, int T, int D,
                      const float* h0, void* h, float* h_out, int* dev_status,
                      la_stream_t stream) {
    if (!scan_shape_ok(B, T, D, dtype)) return LA_ERR_INVALID_ARG;
    if (any_misaligned({x, log_a, h0, h, h_out})) return LA_ERR_INVALID_ARG;
    if (B == 0) return LA_OK;
    const size_t state = (size_t)B * D, n = state * T, es = elem_size(dtype);
    cudaStream_t s = (cudaStream_t)stream;
    if (h0 != h_out && ranges_overlap(h0, state * 4, h_out, state * 4)) return LA_ERR_INVALID_ARG;
    if (T == 0) {  // no token: the final state is the initial one
        if (!h_out) return LA_OK;
        return cuda_status(h0 ? launch_state_copy(h_out, h0, state, s)
                              : launch_state_zero(h_out, nullptr, state, 0, s));
    }
    if (!x || !log_a || !h) return LA_ERR_INVALID_ARG;
    if (clash({{x, n * es}, {log_a, n * 4}}, {{h, n * es}, {h_out, state * 4}}) ||
        ranges_overlap(h, n * es, h0, state * 4))
        return LA_ERR_INVALID_ARG;
    RecurrenceArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.log_a = log_a; a.h0 = h0; a.h = h; a.h_out = h_out;
    a.dev_status = dev_status;
    a.B = B; a.T = T; a.D = D;
    a.bf16 = dtype == LA_DTYPE_BF16;
    return cuda_status(launch_scan_fwd(a, s));
}

la_status la_scan_bwd(const float* log_a, const void* h, const void* dh, la_dtype dtype, int B, int T,
                      int D, const float* h0, const float* dh_T, void* dx, float* dlog_a, float* dh0,
                      int* dev_status, la_stream_t stream) {
    if (!scan_shape_ok(B, T, D, dtype)) return LA_ERR_INVALID_ARG;
    if (any_misaligned({log_a, h, dh, h0, dh_T, dx, dlog_a, dh0})) return LA_ERR_INVALID_ARG;
    if (B == 0) return LA_OK;
    const size_t state = (size_t)B * D, n = state * T, es = elem_size(dtype);
    cudaStream_t s = (cudaStream_t)stream;
    if (dh0 != dh_T && ranges_overlap(dh0, state * 4, dh_T, state * 4)) return LA_ERR_INVALID_ARG;
    if (ranges_overlap(dh0, state * 4, h0, state * 4)) return LA_ERR_INVALID_ARG;
    if (T == 0) {
        if (!dh0) return LA_OK;
        return cuda_status(dh_T ? launch_state_copy(dh0, dh_T, state, s)
                                : launch_state_zero(dh0, nullptr, state, 0, s));
    }
    if (!log_a || !h || !dh || !dx || !dlog_a) return LA_ERR_INVALID_ARG;
    if (clash({{log_a, n * 4}, {h, n * es}, {dh, n * es}, {h0, state * 4}},
              {{dx, n * es}, {dlog_a, n * 4}, {dh0, state * 4}}) ||
        ranges_overlap(dx, n * es, dh_T, state * 4) || ranges_overlap(dlog_a, n * 4, dh_T, state * 4))
        return LA_ERR_INVALID_ARG;
    RecurrenceArgs a;
    std::memset(&a, 0, sizeof(a));
    a.log_a = log_a; a.h = const_cast<void*>(h); a.dh = dh; a.h0 = h0; a.dh_T = dh_T;
    a.dx = dx; a.dlog_a = dlog_a; a.dh0 = dh0;
    a.dev_status = dev_status;
    a.B = B; a.T = T; a.D = D;
    a.bf16 = dtype == LA_DTYPE_BF16;
    return cuda_status(launch_scan_bwd(a, s));
}

la_status la_scan_step(const void* x, la_dtype dtype, const float* log_a, int B, int D,
                       const float* h_in, float* h_out, void* h, la_stream_t stream) {
    if (!scan_shape_ok(B, 1, D, dtype)) return LA_ERR_INVALID_ARG;
    if (any_misaligned({x, log_a, h_in, h_out, h})) return LA_ERR_INVALID_ARG;
    if (B == 0) return LA_OK;
    if (!x || !log_a || !h_in || !h_out || !h) return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)B * D, es = elem_size(dtype);
    if (clash({{x, n * es}, {log_a, n * 4}}, {{h, n * es}, {h_out, n * 4}}) ||
        ranges_overlap(h, n * es, h_in, n * 4) ||
        (h_in != h_out && ranges_overlap(h_in, n * 4, h_out, n * 4)))
        return LA_ERR_INVALID_ARG;
    RecurrenceArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.log_a = log_a; a.h0 = h_in; a.h = h; a.h_out = h_out;
    a.B = B; a.T = 1; a.D = D;
    a.bf16 = dtype == LA_DTYPE_BF16;
    return cuda_status(launch_scan_step(a, (cudaStream_t)stream));
}

}  // extern "C"
