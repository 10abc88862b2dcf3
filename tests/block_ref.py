"""Plain fp64 forms (numpy) of the operators of a state space layer in its residual
block, and the error an fp32 computation of them may make, entry by entry (as in
layer_ref.py: U = 2^-24, roundings counted, magnitudes carried as majorants).

sigma(v) is 1 / (1 + 2^x) with x = -v log2 e rounded (U |x|, and U for the constant): off by
(12 + 4 |v|) U of itself.
"""
import numpy as np

from layer_ref import U


def sigmoid(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def sigmoid_ops(v):
    return 12.0 + 4.0 * np.abs(v)


def silu(v):
    """(v sigma(v), its slope, the slope's rounding in units of U)."""
    s = sigmoid(v)
    slope = s * (1.0 + v * (1.0 - s))
    # 1 - s and the products, each part of the slope with sigma's own error
    ops = (8.0 + 2.0 * sigmoid_ops(v)) * s * (1.0 + np.abs(v))
    return v * s, slope, ops


# ---- short_conv ----------------------------------------------------------------------

def _conv(x, w, bias, state, positions):
    """(u [B,T,D], size, rows [B,T+W-1,D], use [W][B,T,1])."""
    B, T, D = x.shape
    W = w.shape[1]
    rows = np.concatenate((np.zeros((B, W - 1, D)) if state is None else state, x), 1)
    use = [np.ones((B, T, 1), bool) if positions is None or j == W - 1 else (positions >= W - 1 - j)[..., None]
           for j in range(W)]
    u = np.zeros((B, T, D)) if bias is None else np.broadcast_to(bias, (B, T, D)).copy()
    size = np.abs(u)
    for j in range(W):
        term = np.where(use[j], rows[:, j:j + T] * w[:, j], 0.0)
        u, size = u + term, size + np.abs(term)
    return u, size, rows, use


def conv(x, w, bias, act, state, positions):
    """(y, bound, state behind)."""
    u, size, rows, _ = _conv(x, w, bias, state, positions)
    err = (w.shape[1] + 2) * U * size
    if act:
        y, slope, ops = silu(u)
        # the curvature of silu is at most 1/2
        err = err * (np.abs(slope) + err) + (4.0 + sigmoid_ops(u)) * U * np.abs(y)
        u = y
    return u, err, rows[:, x.shape[1]:]


def conv_bwd(x, w, bias, act, state, positions, dy, dstate_T):
    """(dx, bound, dw, bound, db, bound, dstate, bound)."""
    B, T, D = x.shape
    W = w.shape[1]
    u, size, rows, use = _conv(x, w, bias, state, positions)
    du, err = dy, np.zeros_like(dy)
    if act:
        _, slope, ops = silu(u)
        du = dy * slope
        err = np.abs(dy) * ((W + 2) * U * size + (ops + 2.0) * U)
    size = np.abs(du)
    d, db_ = np.zeros(rows.shape), np.zeros(rows.shape)
    if dstate_T is not None:
        d[:, T:] += dstate_T
        db_[:, T:] += (W + 2) * U * np.abs(dstate_T)
    dw, dwb = np.empty((D, W)), np.empty((D, W))
    chain = (16.0 + B * T) * U  # additions a term passes through
    for j in range(W):
        m = use[j]
        d[:, j:j + T] += np.where(m, du * w[:, j], 0.0)
        db_[:, j:j + T] += np.where(m, (err + (W + 2) * U * size) * np.abs(w[:, j]), 0.0)
        at = np.where(m, rows[:, j:j + T], 0.0)
        dw[:, j] = (du * at).sum((0, 1))
        dwb[:, j] = ((err + chain * size) * np.abs(at)).sum((0, 1))
    return (d[:, W - 1:], db_[:, W - 1:], dw, dwb, du.sum((0, 1)), (err + chain * size).sum((0, 1)),
            d[:, :W - 1], db_[:, :W - 1])


# ---- ssm -----------------------------------------------------------------------------

def _heads(v, D):
    B, T, G, N = v.shape
    return np.repeat(v, D // G, axis=2)


def _delta(dt, bias, softplus):
    """(delta, its error relative to itself, slope, the slope's error relative)."""
    v = dt if bias is None else dt + bias
    if not softplus:
        return v, np.full_like(v, 2.0 * U), np.ones_like(v), np.zeros_like(v)
    # the sum's rounding U |v| moves e^v by as much; 2^x of the scaled argument 4 U + 2 U |v|,
    # the polynomial 3 U, the sum U
    return np.logaddexp(v, 0.0), (16.0 + 4.0 * np.abs(v)) * U, sigmoid(v), (sigmoid_ops(v) + 2.0 * np.abs(v)) * U


def _walk(x, dt, A, b, c, bias, softplus, h0, positions):
    B, T, D = x.shape
    N = A.shape[1]
    d, de, slope, slope_e = _delta(dt, bias, softplus)
    bh, ch = _heads(b, D), _heads(c, D)
    h = np.zeros((B, D, N)) if h0 is None else h0.copy()
    m, e = np.abs(h), np.zeros((B, D, N))
    hs, ms, es, a_s = [h], [m], [e], []
    # a sequence cut into chunks joins them by the decay of their sum of delta: that sum is off by
    # T U of itself, and s e^-s is at most 0.37
    cut = 0.4 * T * U
    for t in range(T):
        arg = d[:, t, :, None] * A
        a = np.exp(arg)
        if positions is not None:
            a = np.where((positions[:, t] == 0)[:, None, None], 0.0, a)
        ae = np.abs(arg) * (de[:, t, :, None] + 4.0 * U) + 4.0 * U
        add = (d[:, t] * x[:, t])[..., None] * bh[:, t]
        with np.errstate(invalid="ignore"):
            drop = a == 0.0
            e = np.where(drop, 0.0, a * (e + (ae + 2.0 * U) * m)) + (de[:, t, :, None] + 4.0 * U) * np.abs(add)
            h = np.where(drop, 0.0, a * h) + add
            m = np.where(drop, 0.0, a * m) + np.abs(add)
        e = e + U * m
        hs.append(h), ms.append(m), es.append(e + cut * m), a_s.append((a, ae))
    return d, de, slope, slope_e, bh, ch, hs, ms, es, a_s


def ssm(x, dt, A, b, c, skip, gate, bias, softplus, h0, positions):
    """(y, bound, h_T, bound); b, c [B,T,G,N]."""
    B, T, D = x.shape
    N = A.shape[1]
    _, _, _, _, _, ch, hs, ms, es, _ = _walk(x, dt, A, b, c, bias, softplus, h0, positions)
    u, ub, um = _read(x, skip, ch, hs, ms, es, N)
    if gate is not None:
        act, _, _ = silu(gate)
        ub = np.abs(act) * (ub + (4.0 + sigmoid_ops(gate)) * U * um)
        u = u * act
    return u, ub, hs[-1], es[-1]


def _read(x, skip, ch, hs, ms, es, N):
    T = x.shape[1]
    u, ub, um = (np.empty_like(x) for _ in range(3))
    for t in range(T):
        u[:, t] = (ch[:, t] * hs[t + 1]).sum(-1)
        um[:, t] = (np.abs(ch[:, t]) * ms[t + 1]).sum(-1)
        ub[:, t] = (np.abs(ch[:, t]) * es[t + 1]).sum(-1) + (N + 4) * U * um[:, t]
    if skip is not None:
        u, um = u + skip * x, um + np.abs(skip * x)
        ub = ub + 2.0 * U * um
    return u, ub, um


def ssm_bwd(x, dt, A, b, c, skip, gate, bias, softplus, h0, positions, dy, dh_T):
    """A dict of (gradient, bound): x, dt, A, b, c, skip, gate, bias, h0."""
    B, T, D = x.shape
    G, N = b.shape[2:]
    d, de, slope, slope_e, bh, ch, hs, ms, es, a_s = _walk(x, dt, A, b, c, bias, softplus, h0, positions)
    u, ub, um = _read(x, skip, ch, hs, ms, es, N)
    du, due = dy, np.zeros_like(dy)  # due: relative
    out = {}
    if gate is not None:
        act, gslope, ops = silu(gate)
        out["gate"] = (dy * u * gslope, np.abs(dy) * (ub * np.abs(gslope) + um * (ops + 4.0) * U))
        du, due = dy * act, (4.0 + sigmoid_ops(gate)) * U
    g = np.zeros((B, D, N)) if dh_T is None else dh_T.copy()
    mg, eg = np.abs(g), np.zeros((B, D, N))
    dx, dxb, dd, ddb = (np.empty_like(x) for _ in range(4))
    db, dbb, dc, dcb = (np.empty(b.shape) for _ in range(4))
    dA, dAb = np.zeros_like(A), np.zeros_like(A)
    cut = 0.4 * T * U
    over_channels = (16.0 + D / 8.0) * U   # additions a term of db, dc passes through
    over_tokens = (64.0 + T + B) * U
    group = lambda v: v.reshape(B, G, D // G, N).sum(2)
    for t in range(T - 1, -1, -1):
        a, ae = a_s[t]
        cd = ch[:, t] * du[:, t, :, None]
        g, mg = g + cd, mg + np.abs(cd)
        eg = eg + np.abs(cd) * (np.broadcast_to(due[:, t, :, None], cd.shape) + 2.0 * U) + U * mg
        egc = eg + cut * mg
        into, size = (g * bh[:, t]).sum(-1), (mg * np.abs(bh[:, t])).sum(-1)
        into_e = (egc * np.abs(bh[:, t])).sum(-1) + (N + 4) * U * size
        dxs = (d[:, t] * x[:, t])[..., None]
        db[:, t] = group(g * dxs)
        dbb[:, t] = group(np.abs(dxs) * (egc + mg * (de[:, t, :, None] + 4.0 * U + over_channels)))
        h, m, e = hs[t + 1], ms[t + 1], es[t + 1]
        dus = du[:, t, :, None]
        dc[:, t] = group(h * dus)
        dcb[:, t] = group(np.abs(dus) * (e + m * (np.broadcast_to(due[:, t, :, None], m.shape) + 2.0 * U
                                                  + over_channels)))
        with np.errstate(invalid="ignore"):
            drop = a == 0.0
            q = np.where(drop, 0.0, a * g * hs[t])
            mq = np.where(drop, 0.0, a * mg * ms[t])
            eq = np.where(drop, 0.0, a * (egc * ms[t] + mg * es[t])) + (ae + 4.0 * U) * mq
        along, along_m = (q * A).sum(-1), (mq * np.abs(A)).sum(-1)
        along_e = (eq * np.abs(A)).sum(-1) + (N + 6) * U * along_m
        dA += (q * d[:, t, :, None]).sum(0)
        dAb += ((eq + mq * (de[:, t, :, None] + 2.0 * U + over_tokens)) * np.abs(d[:, t, :, None])).sum(0)
        dx[:, t] = d[:, t] * into
        dxb[:, t] = np.abs(d[:, t]) * (into_e + size * (de[:, t] + 4.0 * U))
        dd[:, t] = x[:, t] * into + along
        ddb[:, t] = np.abs(x[:, t]) * (into_e + 4.0 * U * size) + along_e + 4.0 * U * along_m
        ddb[:, t] = slope[:, t] * (ddb[:, t] + (slope_e[:, t] + 2.0 * U) * (np.abs(x[:, t]) * size + along_m))
        g, mg, eg = a * g, a * mg, a * (eg + (ae + 2.0 * U) * mg)
    dd = dd * slope
    if skip is not None:
        out["skip"] = ((du * x).sum((0, 1)), (np.abs(du * x) * (due + over_tokens)).sum((0, 1)))
        dx, dxb = dx + skip * du, dxb + np.abs(skip * du) * (due + 4.0 * U)
    if bias is not None:
        out["bias"] = (dd.sum((0, 1)), (ddb + over_tokens * np.abs(dd)).sum((0, 1)))
    out.update(x=(dx, dxb), dt=(dd, ddb), A=(dA, dAb), b=(db, dbb), c=(dc, dcb), h0=(g, eg + cut * mg))
    return out


# ---- block_norm ----------------------------------------------------------------------

def _norm(v, eps, center, err=0.0):
    """(normed rows, 1 / root, its error from roundings and from err of v, relative error of the
    root): sums of up to 48 additions, halved by the root, rsqrtf, the products."""
    size = np.abs(v) + (np.abs(v).mean(-1, keepdims=True) if center else 0.0)
    err = err + 48.0 * U * size * (1.0 if center else 0.0)
    if center:
        v = v - v.mean(-1, keepdims=True)
        err = err + np.mean(err, -1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    along = (np.abs(v) * err * np.ones_like(v)).mean(-1, keepdims=True) * r * r
    r_err = along + 32.0 * U
    return v * r, r, err * r + np.abs(v) * r * (r_err + 4.0 * U), r_err


def block(o, h, post, w_post, gate, alpha, beta, pre, w_pre, center, eps):
    """(h', bound, y, bound); gate [D] or [B,1,D] or None, h None: no residual."""
    p, e = o, np.zeros_like(o)
    if post:
        p, _, e, _ = _norm(o, eps, center)
    f = alpha * (1.0 if w_post is None else w_post) * (1.0 if gate is None else gate) * np.ones_like(o)
    out = f * p + (0.0 if h is None else beta * h)
    e = np.abs(f) * (e + 6.0 * U * np.abs(p)) + 2.0 * U * (np.abs(f * p) + (0.0 if h is None else np.abs(beta * h)))
    if not pre:
        return out, e, None, None
    n, _, ne, _ = _norm(out, eps, center, e)
    w = 1.0 if w_pre is None else w_pre
    return out, e, n * w, (ne + 2.0 * U * np.abs(n)) * np.abs(w)


def _norm_bwd(dn, dne, n, ne, r, re, center):
    """(gradient, bound) through the norm for dn with error dne (n with ne, r with re)."""
    dot, dotm = (dn * n).mean(-1, keepdims=True), (np.abs(dn) * np.abs(n)).mean(-1, keepdims=True)
    dot_e = (dne * np.abs(n) + np.abs(dn) * ne).mean(-1, keepdims=True) + 64.0 * U * dotm
    mean = dn.mean(-1, keepdims=True) if center else 0.0
    mean_m = np.abs(dn).mean(-1, keepdims=True) if center else 0.0
    mean_e = (dne.mean(-1, keepdims=True) + 64.0 * U * mean_m) if center else 0.0
    size = np.abs(dn) + mean_m + np.abs(n) * dotm
    return r * (dn - mean - n * dot), r * (dne + mean_e + np.abs(n) * dot_e + ne * np.abs(dot)
                                           + (re + 8.0 * U) * size)


def block_bwd(o, h_out, dy, dh, post, w_post, gate, alpha, beta, pre, w_pre, center, eps):
    """A dict of (gradient, bound): o, h, w_post, gate, w_pre."""
    out = {}
    rows = o.shape[0] * o.shape[1]
    chain = (64.0 + rows) * U
    dt = np.zeros_like(o) if dh is None else dh.copy()
    dte = np.zeros_like(o)
    if pre:
        n, r, ne, re = _norm(h_out, eps, center)
        out["w_pre"] = ((dy * n).sum((0, 1)), (np.abs(dy) * (ne + chain * np.abs(n))).sum((0, 1)))
        w = 1.0 if w_pre is None else w_pre
        back, back_e = _norm_bwd(dy * w, U * np.abs(dy * w), n, ne, r, re, center)
        dte = back_e + 2.0 * U * (np.abs(back) + np.abs(dt))
        dt = dt + back
    out["h"] = (beta * dt, abs(beta) * (dte + 2.0 * U * np.abs(dt)))
    p, pe = o, np.zeros_like(o)
    if post:
        p, r, pe, re = _norm(o, eps, center)
    dt, dte = alpha * dt, abs(alpha) * (dte + 2.0 * U * np.abs(dt))
    wp = 1.0 if w_post is None else w_post
    over = (0, 1) if gate is None or gate.ndim == 1 else 1
    out["gate"] = ((dt * p * wp).sum(over), (np.abs(wp) * (dte * np.abs(p) + np.abs(dt) * (pe + (chain + 4.0 * U)
                                                                                          * np.abs(p)))).sum(over))
    g = 1.0 if gate is None else gate
    dt, dte = dt * g, np.abs(g) * (dte + 2.0 * U * np.abs(dt))
    out["w_post"] = ((dt * p).sum((0, 1)), (dte * np.abs(p) + np.abs(dt) * (pe + (chain + 4.0 * U) * np.abs(p))).sum((0, 1)))
    if post:
        dt, dte = dt * wp, np.abs(wp) * (dte + 2.0 * U * np.abs(dt))
        dt, dte = _norm_bwd(dt, dte, p, pe, r, re, center)
    out["o"] = (dt, dte)
    return out
