"""Plain fp64 forms (numpy) of the operators around retention, and the error an
fp32 computation of them may make, entry by entry.

U = 2^-24 is fp32's unit roundoff.  Every bound below counts roundings: a value
that is the result of n fp32 operations on operands whose sizes add up to m is off
by at most about n U m.  CUDA's documented maximum errors are taken as expf 2 ulp,
rsqrtf 2 ulp, sincospif 2 ulp (1 ulp <= 2 U relative).  `half_step` is what the one
rounding to the output's type adds.
"""
import numpy as np
import torch

U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().to("cpu").double().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(name, got, want, bound, dtype):
    """|got - want| <= bound + half a step of the stored value, entry by entry."""
    got = f64(got)
    assert got.shape == want.shape, f"{name}: {got.shape} for {want.shape}"
    assert np.isfinite(got).all(), f"{name}: not finite"
    limit = bound + half_step(dtype) * (np.abs(want) + bound) + 1e-37
    worst = np.max(np.abs(got - want) / limit) if want.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} of what rounding allows"


# ---- qk_rotate -----------------------------------------------------------------------

def _pairs(rot, interleaved):
    m = np.arange(rot // 2)
    return (2 * m, 2 * m + 1) if interleaved else (m, m + rot // 2)


def turn(x, pos, rot, freq, interleaved, sign=1.0):
    """x [B,T,H,d] turned by pos [B,T] (sign -1: back)."""
    y = np.array(x)
    if rot:
        i, j = _pairs(rot, interleaved)
        ang = (pos[:, :, None].astype(np.float64) * np.asarray(freq, np.float64))[:, :, None]
        c, s = np.cos(ang), sign * np.sin(ang)
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def _pair_size(x, rot, interleaved):
    """|x_i| + |x_j| of each entry's pair, |x| outside the rotated part."""
    m = np.abs(x)
    if rot:
        i, j = _pairs(rot, interleaved)
        m[..., i] = m[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return m


def _angle_error(pos, freq, rot):
    """The angle's error in units of U: the rest of a turn to fp32, and the table's
    64 bits and the reference's own product, 2^-51 of the angle."""
    far = float(np.max(np.abs(pos.astype(np.float64)))) * (float(np.max(np.abs(freq))) if rot else 0.0)
    return 8.0 + far * 2.0 ** -51 / U


def qk(x, pos, rot, freq, interleaved, norm, w, eps, scale):
    """(y [B,H,T,d], bound)."""
    d = x.shape[-1]
    n = x
    if norm:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        n = n if w is None else n * w
    y = scale * turn(n, pos, rot, freq, interleaved)
    # squares and their sum 8 + 5 levels, halved by the root, rsqrtf, products, the turn
    ops = 24.0 + _angle_error(pos, freq, rot)
    bound = ops * U * abs(scale) * _pair_size(n, rot, interleaved)
    return y.transpose(0, 2, 1, 3), bound.transpose(0, 2, 1, 3)


def qk_bwd(x, dy, pos, rot, freq, interleaved, norm, w, eps, scale):
    """(dx [B,T,H,d], bound, dw [d], bound)."""
    g = scale * turn(dy.transpose(0, 2, 1, 3), pos, rot, freq, interleaved, -1.0)
    gm = abs(scale) * _pair_size(dy.transpose(0, 2, 1, 3), rot, interleaved)
    a = _angle_error(pos, freq, rot)
    if not norm:
        return g, (8.0 + a) * U * gm, None, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dw = (g * xh).sum((0, 1, 2))
    chain = min(512, x.shape[0] * x.shape[1] * x.shape[2])  # additions a term passes through
    dwb = (24.0 + a + chain) * U * (gm * np.abs(xh)).sum((0, 1, 2))
    ww = 1.0 if w is None else w
    gx = g * ww
    gxm = gm * np.abs(ww)
    dx = r * (gx - xh * (gx * xh).mean(-1, keepdims=True))
    bound = (48.0 + a) * U * r * (gxm + np.abs(xh) * (gxm * np.abs(xh)).mean(-1, keepdims=True))
    return dx, bound, dw, dwb


# ---- head_gate -----------------------------------------------------------------------

def _norm(o, eps, center):
    """Normed rows, r, and the size of a row entry before the mean is taken out."""
    size = np.abs(o) + (np.abs(o).mean(-1, keepdims=True) if center else 0.0)
    if center:
        o = o - o.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    # entries carry up to 16 U of `size`; r carries their part along the row
    along = (np.abs(o) * size).mean(-1, keepdims=True) * r * r
    err = 16.0 * U * (size * r + np.abs(o) * r * along) + 24.0 * U * np.abs(o) * r
    return o * r, r, err, 16.0 * U * along + 16.0 * U


def gate(o, g, w, eps, center):
    """o [B,H,T,d], g [B,T,H,d], w [H,d] -> (y [B,T,H,d], bound)."""
    n, _, err, _ = _norm(o, eps, center)
    n, err = n.transpose(0, 2, 1, 3), err.transpose(0, 2, 1, 3)
    f = 1.0 if w is None else w
    if g is not None:
        f = f * g / (1.0 + np.exp(-g))
    return n * f, (err + 16.0 * U * np.abs(n)) * np.abs(f) * np.ones_like(n)


def gate_bwd(o, g, dy, w, eps, center):
    """(d_o [B,H,T,d], bound, dg, bound, dw [H,d], bound)."""
    n, r, err, r_err = _norm(o, eps, center)
    n, r, err, r_err = (v.transpose(0, 2, 1, 3) for v in (n, r, err, r_err))
    ww = 1.0 if w is None else w
    du, dum = dy, np.abs(dy)
    dg = dgb = None
    if g is not None:
        s = 1.0 / (1.0 + np.exp(-g))
        slope = s * (1.0 + g * (1.0 - s))
        size = s * (1.0 + np.abs(g) * (1.0 - s))
        # 1 - s: s is off by 8 U of 1
        dg = dy * n * ww * slope
        dgb = np.abs(dy * ww) * (err * np.abs(slope) + np.abs(n) * U * (32.0 * size + 16.0 * np.abs(g) * s))
        du, dum = dy * g * s, np.abs(dy * g * s)
    dw = (du * n).sum((0, 1))
    chain = min(512, o.shape[0] * o.shape[2])
    dwb = (dum * (err + (16.0 + chain) * U * np.abs(n))).sum((0, 1))
    dn, dnm = du * ww, dum * np.abs(ww)
    mean = dn.mean(-1, keepdims=True) if center else 0.0
    meanm = dnm.mean(-1, keepdims=True) if center else 0.0
    dot, dotm = (dn * n).mean(-1, keepdims=True), (dnm * np.abs(n)).mean(-1, keepdims=True)
    dot_err = (dnm * err).mean(-1, keepdims=True) + 32.0 * U * dotm
    d_o = r * (dn - mean - n * dot)
    bound = r * (32.0 * U * (dnm + meanm + np.abs(n) * dotm) + err * np.abs(dot) + np.abs(n) * dot_err
                 + r_err * (dnm + meanm + np.abs(n) * dotm))
    back = lambda v: v.transpose(0, 2, 1, 3)
    return back(d_o), back(bound), dg, dgb, dw, dwb


# ---- scan ----------------------------------------------------------------------------

def scan(x, log_a, h0):
    """(h [B,T,D], bound, h_T, bound): the recurrence token by token beside a majorant
    of its sizes (m) and of the error (e): each step's decay is off by expf's 4 U and a
    rounding, and a term meets about 32 more where runs of tokens are put together.
    A decay that is zero in fp32 restarts its channel."""
    B, T, D = x.shape
    with np.errstate(under="ignore"):
        a = np.exp(log_a)
    a[a < 2.0 ** -150] = 0.0
    h, bound = np.empty_like(x), np.empty_like(x)
    s = np.zeros((B, D)) if h0 is None else h0.copy()
    m, e = np.abs(s), np.zeros((B, D))
    b = np.zeros((B, D))
    for t in range(T):
        at = a[:, t]
        cut = at == 0.0
        with np.errstate(invalid="ignore"):
            e = np.where(cut, 0.0, at * (e + 8.0 * U * m))
            s = np.where(cut, 0.0, at * s) + x[:, t]
            m = np.where(cut, 0.0, at * m) + np.abs(x[:, t])
        b = e + 32.0 * U * m
        h[:, t], bound[:, t] = s, b
    return h, bound, s, b


def scan_bwd(log_a, h, dh, h0, dh_T):
    """(dx, bound, dlog_a, bound, dh0, bound) of the recurrence whose output was h."""
    B, T, D = h.shape
    with np.errstate(under="ignore"):
        a = np.exp(log_a)
    a[a < 2.0 ** -150] = 0.0
    dx, dxb, dla, dlab = (np.empty_like(h) for _ in range(4))
    c = np.zeros((B, D)) if dh_T is None else dh_T.copy()
    m, e = np.abs(c), np.zeros((B, D))
    for t in range(T - 1, -1, -1):
        g, gm = dh[:, t] + c, np.abs(dh[:, t]) + m
        dx[:, t], dxb[:, t] = g, e + 32.0 * U * gm
        c, m, e = a[:, t] * g, a[:, t] * gm, a[:, t] * (e + 8.0 * U * gm)
        prev = h[:, t - 1] if t else (np.zeros((B, D)) if h0 is None else h0)
        cut = a[:, t] == 0.0
        with np.errstate(invalid="ignore"):
            dla[:, t] = np.where(cut, 0.0, c * prev)
            dlab[:, t] = np.where(cut, 0.0, (e + 32.0 * U * m) * np.abs(prev))
    return dx, dxb, dla, dlab, c, e + 32.0 * U * m
