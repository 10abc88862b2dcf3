"""The operators around retention on the host: their plain forms' gradients against
differences, and every refusal of the C ABI and of the binding.

Pointers are fake integers that are never touched: each refused call fails its host
checks, and each accepted one is a call with no tokens and nothing to write.
"""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import layer_ref as ref
import retnet_retention_gb300 as la

FAKE = 0x10000000
MB = 0x100000
BAD = la.LA_ERR_INVALID_ARG
FREQ = (ctypes.c_double * 128)(*[0.5 ** i for i in range(128)])


@pytest.fixture(scope="module")
def lib():
    from retnet_retention_gb300 import _build
    _build.build()
    return la.library()


def s3(*v):
    return None if v == (None,) else (ctypes.c_longlong * 3)(*v)


# ---- the plain forms' gradients against central differences --------------------------

def along(f, x, v, step=1e-6):
    return (f(x + step * v) - f(x - step * v)) / (2 * step)


@pytest.mark.parametrize("interleaved,norm,weight,rot", [(True, True, True, 16), (False, True, False, 32),
                                                         (False, False, False, 16), (True, True, True, 0)])
def test_qk_reference_gradients(interleaved, norm, weight, rot):
    g = np.random.default_rng(1)
    B, T, H, d = 2, 3, 2, 32
    x, dy = g.standard_normal((B, T, H, d)), g.standard_normal((B, H, T, d))
    pos = g.integers(0, 1000, (B, T))
    freq = [10000.0 ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)]
    w = 1 + 0.1 * g.standard_normal(d) if weight else None

    def loss(x, w):
        return (dy * ref.qk(x, pos, rot, freq, interleaved, norm, w, 1e-3, 0.7)[0]).sum()

    dx, _, dw, _ = ref.qk_bwd(x, dy, pos, rot, freq, interleaved, norm, w, 1e-3, 0.7)
    v = g.standard_normal(x.shape)
    assert np.isclose(along(lambda x: loss(x, w), x, v), (dx * v).sum(), rtol=1e-7, atol=1e-7)
    if weight:
        v = g.standard_normal(d)
        assert np.isclose(along(lambda w: loss(x, w), w, v), (dw * v).sum(), rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("gated,weight,center", list(itertools.product([True, False], repeat=3)))
def test_gate_reference_gradients(gated, weight, center):
    g = np.random.default_rng(2)
    B, H, T, d = 2, 3, 2, 16
    o, dy = g.standard_normal((B, H, T, d)) + 0.3, g.standard_normal((B, T, H, d))
    gt = g.standard_normal((B, T, H, d)) if gated else None
    w = 1 + 0.1 * g.standard_normal((H, d)) if weight else None
    loss = lambda o, gt, w: (dy * ref.gate(o, gt, w, 1e-3, center)[0]).sum()
    d_o, _, dg, _, dw, _ = ref.gate_bwd(o, gt, dy, w, 1e-3, center)
    v = g.standard_normal(o.shape)
    assert np.isclose(along(lambda o: loss(o, gt, w), o, v), (d_o * v).sum(), rtol=1e-7, atol=1e-7)
    if gated:
        v = g.standard_normal(gt.shape)
        assert np.isclose(along(lambda q: loss(o, q, w), gt, v), (dg * v).sum(), rtol=1e-7, atol=1e-7)
    if weight:
        v = g.standard_normal(w.shape)
        assert np.isclose(along(lambda w: loss(o, gt, w), w, v), (dw * v).sum(), rtol=1e-7, atol=1e-7)


def test_scan_reference_gradients():
    g = np.random.default_rng(3)
    B, T, D = 2, 9, 4
    x, dh = g.standard_normal((B, T, D)), g.standard_normal((B, T, D))
    log_a, h0, dT = -g.random((B, T, D)), g.standard_normal((B, D)), g.standard_normal((B, D))

    def loss(x, log_a, h0):
        h, _, last, _ = ref.scan(x, log_a, h0)
        return (dh * h).sum() + (dT * last).sum()

    dx, _, dla, _, dh0, _ = ref.scan_bwd(log_a, ref.scan(x, log_a, h0)[0], dh, h0, dT)
    for f, at, grad in ((lambda v: loss(v, log_a, h0), x, dx), (lambda v: loss(x, v, h0), log_a, dla),
                        (lambda v: loss(x, log_a, v), h0, dh0)):
        v = g.standard_normal(at.shape)
        assert np.isclose(along(f, at, v), (grad * v).sum(), rtol=1e-7, atol=1e-7)


# ---- the angle's integer arithmetic --------------------------------------------------

def test_angle_in_integers_keeps_far_positions():
    """p F mod 2^64 with F = round-down(f / 2 pi 2^64): the kernel's angle, in Python
    integers, against the exact product in rationals."""
    from fractions import Fraction
    for f in (1.0, 10000.0 ** (-2 / 128), 10000.0 ** (-126 / 128), 0.0, -0.3, 7.0):
        turns = f * 0.15915494309189533577
        turns -= np.floor(turns)
        F = int(np.ldexp(turns, 64)) if turns < 1.0 else 0
        for p in (0, 1, 77, 2 ** 20 + 1, 2 ** 31 - 1, -1, -(2 ** 31)):
            frac = (p * F) % 2 ** 64
            exact = (Fraction(p) * Fraction(turns)) % 1
            off = abs(Fraction(frac, 2 ** 64) - exact)
            assert min(off, 1 - off) <= Fraction(abs(p), 2 ** 64)
            quarter = ((frac + 2 ** 61) % 2 ** 64) >> 62
            rest = (frac - (quarter << 62)) % 2 ** 64
            rest -= 2 ** 64 if rest >= 2 ** 63 else 0
            ang = (rest >> 32) * 2.0 ** -31 * np.pi
            c, s = np.cos(ang), np.sin(ang)
            cc, ss = (s, c) if quarter & 1 else (c, s)
            cc, ss = (-cc if (quarter + 1) & 2 else cc), (-ss if quarter & 2 else ss)
            want = 2 * np.pi * float(exact)
            tol = 2 ** -28 + abs(p) * 2.0 ** -60
            assert abs(cc - np.cos(want)) <= tol and abs(ss - np.sin(want)) <= tol


# ---- refusals of the C ABI -----------------------------------------------------------

def qk_fwd(lib, **over):
    a = dict(q=FAKE, qs=None, k=FAKE + MB, ks=None, dt=1, B=2, T=3, Hq=4, Hk=2, d=64, rot=64,
             freq=FREQ, pos=None, pos0=0, wq=None, wk=None, eps=1e-6, sq=1.0, sk=1.0,
             flags=la.LA_QK_NORM, yq=FAKE + 2 * MB, yk=FAKE + 3 * MB)
    a.update(over)
    return lib.la_qk_rotate_fwd(a["q"], a["qs"], a["k"], a["ks"], a["dt"], a["B"], a["T"], a["Hq"],
                                a["Hk"], a["d"], a["rot"], a["freq"], a["pos"], a["pos0"], a["wq"],
                                a["wk"], a["eps"], a["sq"], a["sk"], a["flags"], a["yq"], a["yk"], None)


NAN_FREQ = (ctypes.c_double * 32)(float("nan"))

QK_BAD = [
    dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hk=0), dict(Hq=65537), dict(d=0), dict(d=24), dict(d=272),
    dict(rot=-16), dict(rot=8), dict(rot=80), dict(dt=2), dict(flags=4), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(sq=float("nan")), dict(sk=float("inf")),
    dict(freq=None), dict(freq=NAN_FREQ), dict(flags=0, wq=FAKE + 4 * MB), dict(pos0=-1),
    dict(pos0=2 ** 31 - 2), dict(B=65536, T=32768), dict(q=None), dict(k=None), dict(yq=None),
    dict(yk=None), dict(q=FAKE + 2), dict(k=FAKE + MB + 8), dict(yq=FAKE + 2 * MB + 4),
    dict(pos=FAKE + 4 * MB + 4), dict(wq=FAKE + 4 * MB + 8), dict(qs=s3(768, 256, 60)),
    dict(qs=s3(768, -256, 64)), dict(ks=s3(4, 128, 64)), dict(qs=s3(1 << 50, 256, 64)),
    dict(yq=FAKE), dict(yk=FAKE + MB + 16), dict(yk=FAKE + 2 * MB + 16),
    dict(pos=FAKE + 2 * MB), dict(wk=FAKE + 3 * MB),
]


@pytest.mark.parametrize("over", QK_BAD, ids=lambda d: ",".join(d))
def test_qk_rotate_fwd_refuses(lib, over):
    assert qk_fwd(lib, **over) == BAD


def qk_bwd(lib, **over):
    a = dict(q=FAKE, qs=None, k=FAKE + MB, ks=None, gq=FAKE + 2 * MB, gk=FAKE + 3 * MB, dt=1, B=2, T=3,
             Hq=4, Hk=2, d=64, rot=64, freq=FREQ, pos=None, pos0=0, wq=FAKE + 4 * MB, wk=FAKE + 5 * MB,
             eps=1e-6, flags=la.LA_QK_NORM, dq=FAKE + 6 * MB, dqs=None, dk=FAKE + 7 * MB, dks=None,
             dwq=FAKE + 8 * MB, dwk=FAKE + 9 * MB, ws=FAKE + 10 * MB, wb=1 << 20)
    a.update(over)
    return lib.la_qk_rotate_bwd(a["q"], a["qs"], a["k"], a["ks"], a["gq"], a["gk"], a["dt"], a["B"],
                                a["T"], a["Hq"], a["Hk"], a["d"], a["rot"], a["freq"], a["pos"],
                                a["pos0"], a["wq"], a["wk"], a["eps"], 1.0, 1.0, a["flags"], a["dq"],
                                a["dqs"], a["dk"], a["dks"], a["dwq"], a["dwk"], a["ws"], a["wb"], None)


# a packed gradient row of 8 heads of 64: dq in heads 0..3, dk in heads 4..5
ROW = 8 * 64
PACKED = dict(dq=FAKE + 6 * MB, dqs=s3(3 * ROW, ROW, 64), dk=FAKE + 6 * MB + 4 * 64 * 2,
              dks=s3(3 * ROW, ROW, 64))

QK_BWD_BAD = [
    dict(gq=None), dict(gk=None), dict(dq=None), dict(dk=None), dict(gq=FAKE + 2 * MB + 8),
    dict(wq=None), dict(wk=None), dict(ws=None), dict(wb=0), dict(ws=FAKE + 10 * MB + 4),
    dict(dwq=FAKE + 8 * MB + 4), dict(dwk=FAKE + 8 * MB), dict(dq=FAKE), dict(dq=FAKE + 2 * MB),
    dict(dk=FAKE + 6 * MB), dict(dwq=FAKE), dict(ws=FAKE + 3 * MB), dict(ws=FAKE + 6 * MB),
    dict(ws=FAKE + 9 * MB), dict(dqs=s3(768, 256, 0)), dict(dqs=s3(0, 256, 64)),
    dict(dqs=s3(768, 128, 64)), dict(dqs=s3(768, 256, 32)), dict(B=-1), dict(d=20),
    dict(PACKED, dk=FAKE + 6 * MB + 3 * 64 * 2), dict(PACKED, dk=FAKE + 6 * MB + 7 * 64 * 2),
    dict(PACKED, dks=s3(3 * ROW, 2 * ROW, 64)),
]


@pytest.mark.parametrize("over", QK_BWD_BAD, ids=lambda d: ",".join(d))
def test_qk_rotate_bwd_refuses(lib, over):
    assert qk_bwd(lib, **over) == BAD


def gate_call(lib, bwd, **over):
    a = dict(o=FAKE, os=None, g=FAKE + MB, gs=None, dy=FAKE + 2 * MB, dys=None, dt=1, w=FAKE + 3 * MB,
             B=2, H=4, T=3, d=64, flags=0, eps=1e-6, y=FAKE + 4 * MB, ys=None, do=FAKE + 5 * MB, dos=None,
             dg=FAKE + 6 * MB, dgs=None, dw=FAKE + 7 * MB, ws=FAKE + 8 * MB, wb=1 << 20)
    a.update(over)
    if not bwd:
        return lib.la_head_gate_fwd(a["o"], a["os"], a["g"], a["gs"], a["dt"], a["w"], a["B"], a["H"],
                                    a["T"], a["d"], a["flags"], a["eps"], a["y"], a["ys"], None)
    return lib.la_head_gate_bwd(a["o"], a["os"], a["g"], a["gs"], a["dy"], a["dys"], a["dt"], a["w"],
                                a["B"], a["H"], a["T"], a["d"], a["flags"], a["eps"], a["do"], a["dos"],
                                a["dg"], a["dgs"], a["dw"], a["ws"], a["wb"], None)


GATE_BOTH = [dict(B=-1), dict(T=-1), dict(H=0), dict(H=65537), dict(d=8), dict(d=40), dict(d=512),
             dict(dt=-1), dict(flags=2), dict(eps=0.0), dict(eps=float("nan")), dict(B=65536, T=32768),
             dict(o=None), dict(o=FAKE + 8), dict(g=FAKE + MB + 2), dict(w=FAKE + 3 * MB + 8),
             dict(os=s3(768, 192, 20)), dict(gs=s3(768, -64, 64)), dict(os=s3(1 << 60, 192, 64))]
GATE_FWD_BAD = GATE_BOTH + [dict(y=None), dict(y=FAKE + 4 * MB + 8), dict(y=FAKE), dict(y=FAKE + MB),
                            dict(y=FAKE + 3 * MB), dict(ys=s3(768, 256, 0)), dict(ys=s3(768, 128, 64)),
                            dict(ys=s3(512, 256, 64))]
GATE_BWD_BAD = GATE_BOTH + [dict(dy=None), dict(dy=FAKE + 2 * MB + 8), dict(do=None), dict(dg=None),
                            dict(g=None), dict(w=None), dict(ws=None), dict(wb=16), dict(do=FAKE),
                            dict(dg=FAKE + 2 * MB), dict(dw=FAKE + 3 * MB), dict(dg=FAKE + 5 * MB),
                            dict(ws=FAKE + 7 * MB), dict(dw=FAKE + 7 * MB + 4), dict(ws=FAKE + 8 * MB + 8),
                            dict(dos=s3(768, 0, 64)), dict(dgs=s3(0, 256, 64))]


@pytest.mark.parametrize("over", GATE_FWD_BAD, ids=lambda d: ",".join(d))
def test_head_gate_fwd_refuses(lib, over):
    assert gate_call(lib, False, **over) == BAD


@pytest.mark.parametrize("over", GATE_BWD_BAD, ids=lambda d: ",".join(d))
def test_head_gate_bwd_refuses(lib, over):
    assert gate_call(lib, True, **over) == BAD


def scan_call(lib, kind, **over):
    a = dict(x=FAKE, dt=1, la=FAKE + MB, B=2, T=3, D=64, h0=FAKE + 2 * MB, h=FAKE + 3 * MB,
             hT=FAKE + 4 * MB, dh=FAKE + 5 * MB, dT=FAKE + 6 * MB, dx=FAKE + 7 * MB, dla=FAKE + 8 * MB,
             dh0=FAKE + 9 * MB)
    a.update(over)
    if kind == "fwd":
        return lib.la_scan_fwd(a["x"], a["dt"], a["la"], a["B"], a["T"], a["D"], a["h0"], a["h"], a["hT"], None,
                               None)
    if kind == "bwd":
        return lib.la_scan_bwd(a["la"], a["h"], a["dh"], a["dt"], a["B"], a["T"], a["D"], a["h0"], a["dT"],
                               a["dx"], a["dla"], a["dh0"], None, None)
    return lib.la_scan_step(a["x"], a["dt"], a["la"], a["B"], a["D"], a["h0"], a["hT"], a["h"], None)


SCAN_BOTH = [dict(B=-1), dict(D=0), dict(D=8), dict(D=24), dict(dt=2), dict(la=None), dict(h=None),
             dict(la=FAKE + MB + 4), dict(h=FAKE + 3 * MB + 2), dict(h0=FAKE + 2 * MB + 8),
             dict(B=1 << 30), dict(h=FAKE + 2 * MB)]
SCAN_FWD_BAD = SCAN_BOTH + [dict(T=-1), dict(x=None), dict(h=FAKE), dict(h=FAKE + MB), dict(hT=FAKE),
                            dict(hT=FAKE + 3 * MB), dict(hT=FAKE + 2 * MB + 16),
                            dict(B=2 ** 20, T=2 ** 31 - 1)]
SCAN_BWD_BAD = [o for o in SCAN_BOTH if "h" not in o or o["h"] != FAKE + 2 * MB] + [
    dict(T=-1), dict(dh=None), dict(dx=None), dict(dla=None), dict(dx=FAKE + MB), dict(dx=FAKE + 5 * MB),
    dict(dla=FAKE + 3 * MB), dict(dla=FAKE + 7 * MB), dict(dh0=FAKE + 2 * MB), dict(dh0=FAKE + 8 * MB),
    dict(dh0=FAKE + 6 * MB + 16), dict(dx=FAKE + 6 * MB), dict(dT=FAKE + 6 * MB + 4)]
SCAN_STEP_BAD = SCAN_BOTH + [dict(x=None), dict(h0=None), dict(hT=None), dict(hT=FAKE + 2 * MB + 16),
                             dict(h=FAKE), dict(hT=FAKE + MB)]


@pytest.mark.parametrize("kind,over", [(k, o) for k, l in (("fwd", SCAN_FWD_BAD), ("bwd", SCAN_BWD_BAD),
                                                           ("step", SCAN_STEP_BAD)) for o in l],
                         ids=lambda d: d if isinstance(d, str) else ",".join(d))
def test_scan_refuses(lib, kind, over):
    assert scan_call(lib, kind, **over) == BAD


def test_calls_without_tokens_touch_nothing(lib):
    """No tokens: accepted with null tensors, nothing launched where nothing is to be
    written, and no workspace needed."""
    for over in (dict(B=0), dict(T=0)):
        assert qk_fwd(lib, q=None, k=None, yq=None, yk=None, **over) == la.LA_OK
        assert qk_bwd(lib, q=None, k=None, gq=None, gk=None, dq=None, dk=None, dwq=None, dwk=None,
                      ws=None, wb=0, **over) == la.LA_OK
        assert gate_call(lib, False, o=None, y=None, **over) == la.LA_OK
        assert gate_call(lib, True, o=None, do=None, dw=None, ws=None, wb=0, **over) == la.LA_OK
        B, T = over.get("B", 2), over.get("T", 3)
        assert lib.la_qk_rotate_bwd_workspace_size(B, T, 4, 2, 64, 1) == 0
        assert lib.la_head_gate_bwd_workspace_size(B, 4, T, 64, 1) == 0
    assert scan_call(lib, "fwd", B=0) == scan_call(lib, "bwd", B=0) == scan_call(lib, "step", B=0) == la.LA_OK
    assert scan_call(lib, "fwd", T=0, x=None, la=None, h=None, hT=None) == la.LA_OK
    assert scan_call(lib, "bwd", T=0, dx=None, dh0=None) == la.LA_OK


def test_binding_constants_of_the_layer_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "linattn.h")).read()
    defined = {m[0]: int(m[1]) for m in re.findall(r"#define\s+(LA_[A-Z0-9_]+)\s+(\d+)u?\b", text)}
    for name in ("LA_QK_NORM", "LA_QK_ADJACENT", "LA_GATE_CENTER"):
        assert getattr(la, name) == defined[name], name


# ---- refusals of the binding (CPU tensors: nothing reaches the library) ---------------

def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 2, 2, 32)
    for call in (lambda: la.qk_rotate_fwd(q, q), lambda: la.qk_rotate_bwd(q, q, q, q),
                 lambda: la.head_gate_fwd(q), lambda: la.head_gate_bwd(q, None, q),
                 lambda: la.scan_fwd(q[0], q[0]), lambda: la.scan_bwd(q[0], q[0], q[0]),
                 lambda: la.scan_step(q[0, 0], q[0, 0], q[0, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_bad_arguments():
    q = torch.zeros(2, 3, 4, 32)
    for kw, err in ((dict(rot=8), ValueError), (dict(rot=48), ValueError), (dict(inv_freq=[1.0]), ValueError),
                    (dict(positions=torch.zeros(2, 3)), ValueError),
                    (dict(positions=torch.zeros(2, 4, dtype=torch.int32)), ValueError),
                    (dict(pos0=-1), ValueError), (dict(pos0=2 ** 31), ValueError),
                    (dict(q_weight=torch.ones(16)), ValueError),
                    (dict(k_weight=torch.ones(32, dtype=torch.float64)), TypeError)):
        with pytest.raises(err):
            la.qk_rotate_fwd(q, q, **kw)
    with pytest.raises(ValueError):
        la.qk_rotate_fwd(q, torch.zeros(2, 3, 4, 16))
    with pytest.raises(TypeError):
        la.qk_rotate_fwd(q, q.bfloat16())
    with pytest.raises(TypeError):
        la.qk_rotate_fwd(q.half(), q.half())
    with pytest.raises(ValueError, match="one after another"):
        la.qk_rotate_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), q)
    with pytest.raises(ValueError):
        la.head_gate_fwd(q[0])
    with pytest.raises(ValueError):
        la.head_gate_bwd(q, None, q, dgate=q)
    with pytest.raises(ValueError):
        la.scan_fwd(q, q)
    with pytest.raises(ValueError):
        la.scan_step(q[0], q[0], q[0])
    assert la.rotary_frequencies(4) == [1.0, 10000.0 ** -0.5]
    with pytest.raises(ValueError):
        la.rotary_frequencies(3)
