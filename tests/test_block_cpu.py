"""The operators of a state space layer on the host: their plain forms' gradients against
differences, and every refusal of the C ABI and of the binding.

Pointers are fake integers that are never touched: each refused call fails its host
checks, and each accepted one is a call with no tokens and nothing to write.
"""
import ctypes
import itertools
import os
import re

import numpy as np
import pytest
import torch

import block_ref as bref
import retnet_retention_gb300 as la

FAKE = 0x10000000
MB = 0x100000
BAD = la.LA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    from retnet_retention_gb300 import _build
    _build.build()
    return la.library()


def at(k):
    return FAKE + k * MB


def arr(*v):
    return (ctypes.c_longlong * len(v))(*v)


# ---- the plain forms' gradients against central differences --------------------------

def against_differences(loss, where, grads, rng):
    for i, grad in enumerate(grads):
        if grad is None:
            continue
        v = rng.standard_normal(where[i].shape)
        step = lambda s: loss(*[a + s * v if j == i else a for j, a in enumerate(where)])
        slope = (step(1e-6) - step(-1e-6)) / 2e-6
        assert np.isclose(slope, (grad * v).sum(), rtol=1e-6, atol=1e-6), i


@pytest.mark.parametrize("act,positions,state,W", list(itertools.product([True, False], [True, False], [True, False],
                                                                         [2, 4])))
def test_conv_reference_gradients(act, positions, state, W):
    g = np.random.default_rng(1)
    B, T, D = 2, 6, 3
    x, w, b = g.standard_normal((B, T, D)), g.standard_normal((D, W)), g.standard_normal(D)
    s = g.standard_normal((B, W - 1, D)) if state else np.zeros((B, W - 1, D))
    pos = g.integers(-1, 5, (B, T)) if positions else None
    dy, dT = g.standard_normal((B, T, D)), g.standard_normal((B, W - 1, D))

    def loss(x, w, b, s):
        y, _, last = bref.conv(x, w, b, act, s, pos)
        return (dy * y).sum() + (dT * last).sum()

    v = bref.conv_bwd(x, w, b, act, s, pos, dy, dT)
    against_differences(loss, [x, w, b, s], [v[0], v[2], v[4], v[6]], g)


@pytest.mark.parametrize("softplus,positions", list(itertools.product([True, False], repeat=2)))
def test_ssm_reference_gradients(softplus, positions):
    g = np.random.default_rng(2)
    B, T, D, N, G = 2, 5, 4, 3, 2
    r = g.standard_normal
    x, dt, A = r((B, T, D)), r((B, T, D)) if softplus else g.random((B, T, D)), -g.random((D, N))
    b, c, skip, gate, bias, h0 = r((B, T, G, N)), r((B, T, G, N)), r(D), r((B, T, D)), r(D) * 0.3, r((B, D, N))
    pos = g.integers(0, 3, (B, T)) if positions else None
    dy, dh = r((B, T, D)), r((B, D, N))

    def loss(x, dt, A, b, c, skip, gate, bias, h0):
        y, _, h, _ = bref.ssm(x, dt, A, b, c, skip, gate, bias, softplus, h0, pos)
        return (dy * y).sum() + (dh * h).sum()

    v = bref.ssm_bwd(x, dt, A, b, c, skip, gate, bias, softplus, h0, pos, dy, dh)
    names = ("x", "dt", "A", "b", "c", "skip", "gate", "bias", "h0")
    against_differences(loss, [x, dt, A, b, c, skip, gate, bias, h0], [v[n][0] for n in names], g)


@pytest.mark.parametrize("post,pre,center,each", list(itertools.product([True, False], repeat=4)))
def test_block_reference_gradients(post, pre, center, each):
    g = np.random.default_rng(3)
    B, T, D = 2, 3, 8
    r = g.standard_normal
    o, h, wp, wq = r((B, T, D)) + 0.3, r((B, T, D)), 1 + 0.1 * r(D), 1 + 0.1 * r(D)
    gate = r((B, 1, D)) if each else r(D)
    dy, dh = r((B, T, D)), r((B, T, D))

    def loss(o, h, wp, gate, wq):
        out = bref.block(o, h, post, wp if post else None, gate, 0.7, 1.5, pre, wq, center, 1e-3)
        return (out[0] * dh).sum() + ((out[2] * dy).sum() if pre else 0.0)

    h_out = bref.block(o, h, post, wp if post else None, gate, 0.7, 1.5, pre, wq, center, 1e-3)[0]
    v = bref.block_bwd(o, h_out, dy, dh, post, wp if post else None, gate, 0.7, 1.5, pre, wq, center, 1e-3)
    dg = v["gate"][0][:, None] if each else v["gate"][0]
    against_differences(loss, [o, h, wp, gate, wq],
                        [v["o"][0], v["h"][0], v["w_post"][0] if post else None, dg, v["w_pre"][0] if pre else None], g)


def test_log1p_polynomial():
    """The kernel's coefficients, in fp32 with fused steps: 3 U of log(1 + p)."""
    src = open(os.path.join(os.path.dirname(la.__file__), "csrc", "ssm.cuh")).read()
    body = src[src.index("k[9] = {"):]
    body = body[:body.index("};")]
    c = [np.float32(m) for m in re.findall(r"(-?\d+\.\d+)f", body)]
    assert len(c) == 9
    p = np.concatenate((np.linspace(0, 1, 100001), 2.0 ** -np.arange(1, 120.0))).astype(np.float32)
    q = np.full_like(p, c[0])
    for a in c[1:]:
        q = np.float32(q.astype(np.float64) * p + a)
    got = (q * p).astype(np.float64)
    want = np.log1p(p.astype(np.float64))
    assert (np.abs(got - want) <= 3 * 2.0 ** -24 * want).all()


# ---- refusals of the C ABI -----------------------------------------------------------

def conv_call(lib, kind, **over):
    a = dict(x=at(0), xs=None, dt=1, w=at(1), b=at(2), B=2, T=3, D=64, W=4, flags=1, s=at(3), pos=None, y=at(4), ys=None,
             so=at(5), dy=at(6), dys=None, dT=at(7), dx=at(8), dxs=None, dw=at(9), db=at(10), ds=at(11), ws=at(12),
             wb=1 << 20, x1=64)
    a.update(over)
    if kind == "fwd":
        return lib.la_short_conv_fwd(a["x"], a["xs"], a["dt"], a["w"], a["b"], a["B"], a["T"], a["D"], a["W"], a["flags"],
                                     a["s"], a["pos"], a["y"], a["ys"], a["so"], None)
    if kind == "bwd":
        return lib.la_short_conv_bwd(a["x"], a["xs"], a["dy"], a["dys"], a["dt"], a["w"], a["b"], a["B"], a["T"], a["D"],
                                     a["W"], a["flags"], a["s"], a["pos"], a["dT"], a["dx"], a["dxs"], a["dw"], a["db"],
                                     a["ds"], a["ws"], a["wb"], None)
    return lib.la_short_conv_step(a["x"], a["x1"], a["dt"], a["w"], a["b"], a["B"], a["D"], a["W"], a["flags"], a["s"],
                                  a["so"], a["y"], None)


CONV_ALL = [dict(B=-1), dict(D=0), dict(D=24), dict(W=1), dict(W=5), dict(dt=2), dict(flags=2), dict(x=None), dict(w=None),
            dict(x=FAKE + 8), dict(w=at(1) + 4), dict(b=at(2) + 8), dict(s=at(3) + 2), dict(B=1 << 30)]
CONV_FWD = CONV_ALL + [dict(T=-1), dict(y=None), dict(y=at(4) + 8), dict(y=at(0)), dict(y=at(1)), dict(y=at(2)),
                       dict(y=at(3)), dict(so=at(4) + 16), dict(so=at(3) + 16), dict(so=at(0)), dict(so=at(5) + 4),
                       dict(pos=at(6) + 4), dict(pos=at(4)), dict(xs=arr(192, 60)), dict(xs=arr(-192, 64)),
                       dict(ys=arr(192, 32)), dict(ys=arr(0, 64)), dict(xs=arr(1 << 50, 64)), dict(B=65536, T=32768), dict(B=1, T=2 ** 31 - 255)]
CONV_BWD = CONV_ALL + [dict(T=-1), dict(dy=None), dict(dx=None), dict(dx=at(0)), dict(dx=at(6)), dict(dx=at(7)),
                       dict(dw=at(1)), dict(dw=at(10)), dict(db=at(2)), dict(ds=at(3)), dict(ds=at(7)), dict(ds=at(8)),
                       dict(ws=None), dict(wb=0), dict(ws=at(12) + 8), dict(ws=at(0)), dict(ws=at(9)), dict(dw=at(9) + 4),
                       dict(dxs=arr(192, 32)), dict(dys=arr(192, 4)), dict(dT=at(7) + 8)]
CONV_STEP = CONV_ALL + [dict(s=None), dict(so=None), dict(y=None), dict(y=at(0)), dict(y=at(3)), dict(so=at(3) + 16),
                        dict(so=at(4)), dict(x1=60), dict(x1=-64)]


@pytest.mark.parametrize("kind,over", [(k, o) for k, l in (("fwd", CONV_FWD), ("bwd", CONV_BWD), ("step", CONV_STEP))
                                       for o in l], ids=lambda d: d if isinstance(d, str) else ",".join(d))
def test_short_conv_refuses(lib, kind, over):
    assert conv_call(lib, kind, **over) == BAD


def ssm_call(lib, kind, **over):
    a = dict(x=at(0), dt=at(1), A=at(2), b=at(3), c=at(4), k=at(5), g=at(6), bias=at(7), st=None, ty=1, B=2, T=3, D=64,
             N=16, G=2, flags=1, h0=at(8), pos=None, y=at(9), h=at(10), ws=at(11), wb=1 << 30, dy=at(12), dT=at(13),
             dx=at(14), ddt=at(15), dA=at(16), db=at(17), dc=at(18), dk=at(19), dg=at(20), dbias=at(21), dh0=at(22))
    a.update(over)
    front = [a[n] for n in ("x", "dt", "A", "b", "c", "k", "g", "bias")]
    if kind == "fwd":
        return lib.la_ssm_fwd(*front, a["st"], a["ty"], a["B"], a["T"], a["D"], a["N"], a["G"], a["flags"], a["h0"],
                              a["pos"], a["y"], a["h"], a["ws"], a["wb"], None)
    if kind == "bwd":
        return lib.la_ssm_bwd(*front, a["dy"], a["st"], a["ty"], a["B"], a["T"], a["D"], a["N"], a["G"], a["flags"],
                              a["h0"], a["pos"], a["dT"], a["dx"], a["ddt"], a["dA"], a["db"], a["dc"], a["dk"], a["dg"],
                              a["dbias"], a["dh0"], a["ws"] if "ws" in over else at(30), a["wb"], None)
    return lib.la_ssm_step(*front, a["st"], a["ty"], a["B"], a["D"], a["N"], a["G"], a["flags"], a["h0"], a["h"], a["y"],
                           None)


def pairs(count, **over):
    """Dense pairs for 2 x 3 tokens of 64 channels and 2 x 16 shared, some replaced."""
    width = [64, 64, 32, 32, 64] + ([64] if count == 6 else [64, 64, 64, 32, 32, 64] if count == 11 else [])
    v = [[3 * w, w] for w in width]
    for k, p in over.items():
        v[int(k[1:])] = list(p)
    return arr(*[s for p in v for s in p])


SSM_ALL = [dict(B=-1), dict(B=65536), dict(D=0), dict(D=24), dict(N=4), dict(N=12), dict(N=128), dict(G=0), dict(G=3), dict(G=16), dict(D=524288, G=65536),
           dict(ty=2), dict(flags=2), dict(x=None), dict(dt=None), dict(A=None), dict(b=None), dict(c=None),
           dict(x=at(0) + 8), dict(A=at(2) + 4), dict(b=at(3) + 2), dict(k=at(5) + 4), dict(bias=at(7) + 8),
           dict(g=at(6) + 8), dict(h0=at(8) + 4)]
SSM_FWD = SSM_ALL + [dict(T=-1), dict(B=1, T=2 ** 31 - 255), dict(y=None), dict(y=at(0)), dict(y=at(3)), dict(y=at(2)), dict(h=at(8) + 16), dict(h=at(9)),
                     dict(h=at(10) + 4), dict(y=at(9) + 2), dict(pos=at(9)), dict(pos=at(23) + 4),
                     dict(st=pairs(6, _0=(192, 60))), dict(st=pairs(6, _2=(96, -32))), dict(st=pairs(6, _5=(192, 32))),
                     dict(st=pairs(6, _5=(0, 64))), dict(st=pairs(6, _4=(1 << 50, 64)))]
SSM_BWD = SSM_ALL + [dict(T=-1), dict(dy=None), dict(dx=None), dict(ddt=None), dict(db=None), dict(dc=None), dict(dg=None),
                     dict(g=None), dict(dx=at(0)), dict(ddt=at(1)), dict(db=at(4)), dict(dA=at(2)), dict(dk=at(5)),
                     dict(dbias=at(19)), dict(dh0=at(13)), dict(dh0=at(8)), dict(dx=at(15)), dict(ws=None), dict(wb=0),
                     dict(ws=at(0)), dict(ws=at(30) + 8), dict(st=pairs(11, _6=(192, 32))), dict(st=pairs(11, _8=(96, 16))),
                     dict(st=pairs(11, _5=(192, 3))), dict(dA=at(16) + 8), dict(dT=at(13) + 4)]
SSM_STEP = SSM_ALL + [dict(h0=None), dict(h=None), dict(y=None), dict(y=at(0)), dict(y=at(8)), dict(h=at(8) + 16),
                      dict(h=at(0)), dict(st=arr(60, 64, 32, 32, 64)), dict(st=arr(64, 64, -32, 32, 64))]


@pytest.mark.parametrize("kind,over", [(k, o) for k, l in (("fwd", SSM_FWD), ("bwd", SSM_BWD), ("step", SSM_STEP))
                                       for o in l], ids=lambda d: d if isinstance(d, str) else ",".join(d))
def test_ssm_refuses(lib, kind, over):
    assert ssm_call(lib, kind, **over) == BAD


def block_call(lib, bwd, **over):
    a = dict(o=at(0), os=None, ty=1, h=at(1), hs=None, rty=0, wp=at(2), g=at(3), wq=at(4), B=2, T=3, D=64, flags=3, al=1.0,
             be=1.0, eps=1e-6, ho=at(5), hos=None, y=at(6), ys=None, dy=at(7), dh=at(8), d_o=at(9), dr=at(10), drs=None,
             dwp=at(11), dg=at(12), dwq=at(13), ws=at(14), wb=1 << 20, dos=None)
    a.update(over)
    if not bwd:
        return lib.la_block_norm_fwd(a["o"], a["os"], a["ty"], a["h"], a["hs"], a["rty"], a["wp"], a["g"], a["wq"], a["B"],
                                     a["T"], a["D"], a["flags"], a["al"], a["be"], a["eps"], a["ho"], a["hos"], a["y"],
                                     a["ys"], None)
    return lib.la_block_norm_bwd(a["o"], a["os"], a["ty"], a["ho"], a["hos"], a["rty"], a["dy"], None, a["dh"], None,
                                 a["wp"], a["g"], a["wq"], a["B"], a["T"], a["D"], a["flags"], a["al"], a["be"], a["eps"],
                                 a["d_o"], a["dos"], a["dr"], a["drs"], a["dwp"], a["dg"], a["dwq"], a["ws"], a["wb"], None)


BLOCK_ALL = [dict(B=-1), dict(B=65536), dict(T=-1), dict(D=0), dict(D=24), dict(D=8208), dict(ty=2), dict(rty=2),
             dict(ty=0, rty=1), dict(flags=16), dict(flags=2), dict(flags=1), dict(flags=11, g=None), dict(al=float("nan")),
             dict(be=float("inf")), dict(eps=0.0), dict(eps=float("nan")), dict(o=None), dict(o=at(0) + 8),
             dict(wp=at(2) + 4), dict(g=at(3) + 8), dict(wq=at(4) + 4), dict(os=arr(192, 60)), dict(os=arr(192, -64)),
             dict(B=32768, T=65536), dict(B=1, T=2 ** 31 - 255)]
BLOCK_FWD = BLOCK_ALL + [dict(y=None), dict(flags=1, wq=None, ho=None, y=None), dict(h=at(1) + 8), dict(ho=at(5) + 4),
                         dict(y=at(0)), dict(y=at(1)), dict(y=at(5)), dict(ho=at(0)), dict(ho=at(1) + 64), dict(y=at(2)),
                         dict(hos=arr(192, 32)), dict(ys=arr(0, 64)), dict(ho=at(1), hos=arr(256, 64)), dict(ho=at(3))]
BLOCK_BWD = BLOCK_ALL + [dict(dy=None), dict(ho=None), dict(d_o=None), dict(d_o=at(0)), dict(dr=at(9)), dict(dr=at(8) + 16),
                         dict(dr=at(5)), dict(dwp=at(2)), dict(dwp=at(13)), dict(ws=None), dict(wb=0), dict(ws=at(14) + 4),
                         dict(ws=at(9)), dict(dos=arr(192, 32)), dict(drs=arr(0, 64)), dict(g=None), dict(wp=None),
                         dict(wq=None), dict(dg=at(12) + 4), dict(dh=at(8) + 4)]


@pytest.mark.parametrize("bwd,over", [(b, o) for b, l in ((False, BLOCK_FWD), (True, BLOCK_BWD)) for o in l],
                         ids=lambda d: str(d) if isinstance(d, bool) else ",".join(d))
def test_block_norm_refuses(lib, bwd, over):
    assert block_call(lib, bwd, **over) == BAD


def test_calls_without_tokens_touch_nothing(lib):
    none = dict(x=None, y=None, so=None, dy=None, dx=None, dw=None, db=None, ds=None, ws=None, wb=0)
    for over in (dict(B=0), dict(T=0)):
        B, T = over.get("B", 2), over.get("T", 3)
        assert conv_call(lib, "fwd", **none, **over) == conv_call(lib, "bwd", **none, **over) == la.LA_OK
        assert lib.la_short_conv_bwd_workspace_size(B, T, 64, 4, 1) == 0
        assert lib.la_ssm_workspace_size(B, T, 64, 16, 1, 1) == lib.la_ssm_bwd_workspace_size(B, T, 64, 16, 1, 1) == 0
        assert lib.la_block_norm_bwd_workspace_size(B, T, 64, 1, 3) == 0
        gone = dict(x=None, dt=None, b=None, c=None, y=None, h=None, dy=None, dx=None, ddt=None, dA=None, db=None, dc=None,
                    dk=None, dg=None, dbias=None, dh0=None, ws=None, wb=0)
        assert ssm_call(lib, "fwd", **gone, **over) == ssm_call(lib, "bwd", **gone, **over) == la.LA_OK
        assert block_call(lib, False, o=None, ho=None, y=None, **over) == la.LA_OK
        assert block_call(lib, True, o=None, d_o=None, dr=None, dwp=None, dg=None, dwq=None, ws=None, wb=0, **over) == la.LA_OK
    assert conv_call(lib, "step", B=0, **none) == ssm_call(lib, "step", B=0) == la.LA_OK


def test_workspaces_are_asked_for_sizes_that_hold(lib):
    """0 for what a call would refuse; more where there is more to keep."""
    for bad in ((2, 9, 24, 16, 1, 1), (2, 9, 64, 7, 1, 1), (2, 9, 64, 16, 3, 1), (2, 9, 64, 16, 1, 5), (-1, 9, 64, 16, 1, 1)):
        assert lib.la_ssm_workspace_size(*bad) == lib.la_ssm_bwd_workspace_size(*bad) == 0
    assert lib.la_short_conv_bwd_workspace_size(2, 9, 64, 5, 1) == lib.la_block_norm_bwd_workspace_size(2, 9, 24, 1, 2) == 0
    small, large = (lib.la_ssm_bwd_workspace_size(2, T, 64, 16, 1, 1) for T in (64, 640))
    assert 0 < small < large


def test_binding_constants_of_the_block_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "linattn.h")).read()
    defined = {m[0]: int(m[1]) for m in re.findall(r"#define\s+(LA_[A-Z0-9_]+)\s+(\d+)u?\b", text)}
    for name in ("LA_CONV_SILU", "LA_SSM_SOFTPLUS", "LA_BLOCK_POST_NORM", "LA_BLOCK_PRE_NORM", "LA_BLOCK_CENTER",
                 "LA_BLOCK_GATE_EACH"):
        assert getattr(la, name) == defined[name], name


# ---- refusals of the binding (CPU tensors: nothing reaches the library) ---------------

X, WT, S = torch.zeros(2, 3, 32), torch.zeros(32, 4), torch.zeros(2, 3, 32)
A, BC, H = torch.zeros(32, 8), torch.zeros(2, 3, 8), torch.zeros(2, 32, 8)


def test_binding_refuses_host_tensors():
    for call in (lambda: la.short_conv_fwd(X, WT), lambda: la.short_conv_bwd(X, WT, X),
                 lambda: la.short_conv_step(X[:, 0], WT, S), lambda: la.ssm_fwd(X, X, A, BC, BC),
                 lambda: la.ssm_bwd(X, X, A, BC, BC, X), lambda: la.ssm_step(X[:, 0], X[:, 0], A, BC[:, 0], BC[:, 0], H),
                 lambda: la.block_norm_fwd(X, X), lambda: la.block_norm_bwd(X, X, X)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_bad_arguments():
    half = X.half()
    value = [lambda: la.short_conv_fwd(X[0], WT), lambda: la.short_conv_fwd(X, torch.zeros(16, 4)),
             lambda: la.short_conv_fwd(X, torch.zeros(32, 5)), lambda: la.short_conv_fwd(X, torch.zeros(32, 1)),
             lambda: la.short_conv_fwd(X, WT, bias=torch.zeros(16)), lambda: la.short_conv_step(X, WT, S),
             lambda: la.short_conv_step(torch.zeros(32, 2).t(), WT, S),
             lambda: la.ssm_fwd(X, X, torch.zeros(32, 12), BC, BC), lambda: la.ssm_fwd(X, X[:, :2], A, BC, BC),
             lambda: la.ssm_fwd(X, X, A, BC, BC[:, :2]), lambda: la.ssm_fwd(X, X, A, torch.zeros(2, 3, 3, 8),
                                                                            torch.zeros(2, 3, 3, 8)),
             lambda: la.ssm_fwd(X, X, A, torch.zeros(2, 3, 16), torch.zeros(2, 3, 16)),
             lambda: la.ssm_fwd(X, X, A, torch.zeros(2, 2, 8), torch.zeros(2, 2, 8)),
             lambda: la.ssm_fwd(X, X, A, BC, BC, gate=X[:, :, :16]), lambda: la.ssm_fwd(X, X, A, BC, BC, skip=A),
             lambda: la.ssm_bwd(X, X, A, BC, BC, X, dgate=X), lambda: la.ssm_step(X, X, A, BC, BC, H),
             lambda: la.block_norm_fwd(X[0], X[0]), lambda: la.block_norm_fwd(X, X, post_weight=A[:, 0]),
             lambda: la.block_norm_fwd(X, X, pre_norm=False, pre_weight=A[:, 0]),
             lambda: la.block_norm_fwd(X, X, gate=torch.zeros(3, 32)), lambda: la.block_norm_fwd(X, X, pre_norm=False, out=X),
             lambda: la.block_norm_bwd(X, X, None), lambda: la.block_norm_bwd(X, X, X, pre_norm=False)]
    kind = [lambda: la.short_conv_fwd(half, WT), lambda: la.short_conv_fwd(X, WT.double()),
            lambda: la.ssm_fwd(X, X.bfloat16(), A, BC, BC), lambda: la.ssm_fwd(X, X, A.double(), BC, BC),
            lambda: la.ssm_fwd(X, X, A, BC.bfloat16(), BC), lambda: la.block_norm_fwd(half, half),
            lambda: la.block_norm_fwd(X, X.bfloat16())]
    for calls, err in ((value, ValueError), (kind, TypeError)):
        for k, call in enumerate(calls):
            with pytest.raises(err):
                call()
                pytest.fail(f"call {k} passed")
