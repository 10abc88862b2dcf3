"""short_conv_fwd, _bwd and _step against the sum over taps in fp64 (GPU)."""
import pytest
import torch

import block_ref as bref
import layer_ref as ref

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


# B, T, D, W, type, activation, bias, state, positions, x a slice of a wider row
CASES = [
    (1, 1, 16, 4, "f32", True, True, True, False, False),
    (1, 1, 32, 2, "bf16", True, False, False, False, True),
    (2, 2, 48, 4, "bf16", False, True, True, True, False),
    (3, 3, 16, 4, "f32", True, True, True, False, True),
    (2, 4, 80, 3, "bf16", True, False, True, True, True),
    (3, 7, 64, 4, "f32", True, True, False, True, False),
    (2, 8, 208, 2, "bf16", True, True, True, True, False),
    (1, 9, 272, 4, "f32", False, False, True, False, False),
    (5, 63, 112, 3, "f32", True, True, True, True, True),
    (2, 64, 528, 4, "bf16", True, True, True, True, True),
    (1, 65, 4096, 4, "bf16", True, True, False, False, False),
    (3, 200, 1040, 4, "f32", True, False, True, True, False),
    (2, 1021, 256, 4, "bf16", True, True, True, True, True),
    (37, 130, 48, 2, "bf16", True, True, False, True, False),
    (1, 5003, 16, 4, "bf16", True, True, True, True, False),
    (4, 700, 2064, 4, "bf16", True, True, True, False, True),
]


def inputs(c, seed=0):
    B, T, D, W, dt, act, bias, state, positions, sliced = c
    g = torch.Generator().manual_seed(seed + B + 7 * T + 11 * D + 13 * W)
    ty = TYPES[dt]
    to = lambda t: t.to(DEV)
    x = to(torch.randn(B, T, 2 * D if sliced else D, generator=g).to(ty))
    x = x[..., D:] if sliced else x
    w = to(torch.randn(D, W, generator=g) * 0.5)
    b = to(torch.randn(D, generator=g)) if bias else None
    s = to(torch.randn(B, W - 1, D, generator=g).to(ty)) if state else None
    pos = None
    if positions:  # short documents, each token its place, some places below 0
        start = torch.rand(B, T, generator=g) < 0.2
        at = torch.arange(T).expand(B, T)
        first = torch.where(start, at, torch.full_like(at, -9 if state else 0)).cummax(1).values
        pos = to((at - first).to(torch.int32))
        pos[:, T // 2] = -5
    dy = to(torch.randn(B, T, D, generator=g).to(ty))
    dT = to(torch.randn(B, W - 1, D, generator=g).to(ty)) if state else None
    return x, w, b, s, pos, dy, dT


def plain(t):
    return None if t is None else ref.f64(t)


ids = lambda c: "x".join(map(str, c))


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_forward(c):
    x, w, b, s, pos, _, _ = inputs(c)
    y, last = la.short_conv_fwd(x, w, bias=b, silu=c[5], state=s, positions=pos)
    torch.cuda.synchronize()
    want, bound, tail = bref.conv(plain(x), plain(w), plain(b), c[5], plain(s), None if pos is None else pos.cpu().numpy())
    ref.check("y", y, want, bound, x.dtype)
    assert (ref.f64(last) == tail).all()


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_backward(c):
    x, w, b, s, pos, dy, dT = inputs(c)
    dx, dw, db, ds = la.short_conv_bwd(x, w, dy, bias=b, silu=c[5], state=s, positions=pos, dstate_T=dT)
    torch.cuda.synchronize()
    v = bref.conv_bwd(plain(x), plain(w), plain(b), c[5], plain(s), None if pos is None else pos.cpu().numpy(),
                      plain(dy), plain(dT))
    ref.check("dx", dx, v[0], v[1], x.dtype)
    ref.check("dweight", dw, v[2], v[3], torch.float32)
    assert (db is None) == (b is None)
    if b is not None:
        ref.check("dbias", db, v[4], v[5], torch.float32)
    ref.check("dstate", ds, v[6], v[7], x.dtype)


@pytest.mark.parametrize("B,D,W,dt,sliced", [(1, 16, 4, "f32", False), (3, 48, 2, "bf16", True), (256, 4096, 4, "bf16", True),
                                             (5, 1040, 3, "f32", True)])
def test_step(B, D, W, dt, sliced):
    """A step is a call of one token: in place or not."""
    x, w, b, s, _, _, _ = inputs((B, 1, D, W, dt, True, True, True, False, sliced))
    y, last = la.short_conv_fwd(x, w, bias=b, state=s)
    new = torch.empty_like(s)
    y2 = la.short_conv_step(x[:, 0], w, s, bias=b, state_out=new)
    s1 = s.clone()
    y1 = la.short_conv_step(x[:, 0], w, s1, bias=b)
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and torch.equal(s1, new) and torch.equal(new, last)
    want, bound, _ = bref.conv(plain(x), plain(w), plain(b), True, plain(s), None)
    ref.check("y", y1.unsqueeze(1), want, bound, x.dtype)


@pytest.mark.parametrize("T,cut", [(6, 1), (6, 2), (150, 64), (150, 3)])
def test_calls_continue_each_other(T, cut):
    x, w, b, s, _, _, _ = inputs((2, T, 48, 4, "bf16", True, True, True, False, False))
    want, tail = la.short_conv_fwd(x, w, bias=b, state=s)
    st = s.clone()
    y1, _ = la.short_conv_fwd(x[:, :cut], w, bias=b, state=st, state_out=st)
    y2, _ = la.short_conv_fwd(x[:, cut:], w, bias=b, state=st, state_out=st)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat((y1, y2), 1), want) and torch.equal(st, tail)


def test_what_does_not_count_does_not_pass():
    """NaN and infinities of one document reach nothing of the next, forward or backward."""
    x, w, b, s, _, dy, _ = inputs((2, 100, 64, 4, "f32", True, True, True, False, False))
    cut = 41
    pos = torch.cat((torch.arange(cut) + 9, torch.arange(100 - cut))).to(torch.int32).expand(2, -1).contiguous().to(DEV)
    clean, _ = la.short_conv_fwd(x, w, bias=b, state=s, positions=pos)
    bad = x.clone()
    bad[:, :cut, ::2], bad[:, :cut, 1::4] = float("nan"), float("inf")
    y, _ = la.short_conv_fwd(bad, w, bias=b, state=torch.full_like(s, float("nan")), positions=pos)
    torch.cuda.synchronize()
    assert torch.equal(y[:, cut:], clean[:, cut:])
    want = la.short_conv_bwd(x, w, dy, bias=b, state=s, positions=pos)
    bad_dy = dy.clone()
    bad_dy[:, cut:] = float("nan")
    got = la.short_conv_bwd(x, w, bad_dy, bias=b, state=s, positions=pos)
    torch.cuda.synchronize()
    assert torch.equal(got[0][:, :cut], want[0][:, :cut]) and torch.equal(got[3], want[3])


def test_outputs_end_where_they_end():
    c = (3, 77, 80, 4, "bf16", True, True, True, False, False)
    x, w, b, s, _, dy, dT = inputs(c)
    B, T, D = x.shape
    row = torch.full((B, T, 3 * D), 3.0, dtype=x.dtype, device=DEV)
    want, _ = la.short_conv_fwd(x, w, bias=b, state=s)
    la.short_conv_fwd(x, w, bias=b, state=s, out=row[..., D:2 * D])
    wx = la.short_conv_bwd(x, w, dy, bias=b, state=s, dstate_T=dT)[0]
    grad = torch.full((B, T, 3 * D), 3.0, dtype=x.dtype, device=DEV)
    la.short_conv_bwd(x, w, dy, bias=b, state=s, dstate_T=dT, dx=grad[..., D:2 * D])
    torch.cuda.synchronize()
    for t, v in ((row, want), (grad, wx)):
        assert torch.equal(t[..., D:2 * D], v)
        assert bool((t[..., :D] == 3).all()) and bool((t[..., 2 * D:] == 3).all())


def test_no_tokens():
    x = torch.zeros(2, 0, 32, device=DEV)
    w, s = torch.ones(32, 4, device=DEV), torch.randn(2, 3, 32, device=DEV)
    y, last = la.short_conv_fwd(x, w, state=s)
    assert y.shape == (2, 0, 32) and torch.equal(last, s)
    assert bool((la.short_conv_fwd(x, w)[1] == 0).all())
    dx, dw, db, ds = la.short_conv_bwd(x, w, x, bias=w[:, 0].contiguous(), state=s, dstate_T=s)
    assert bool((dw == 0).all()) and bool((db == 0).all()) and torch.equal(ds, s)
    assert bool((la.short_conv_bwd(x, w, x)[3] == 0).all())


def test_offsets_past_2_31_elements():
    """A constant input: every token behind the third is the sum of the taps."""
    T, D = 2 ** 20 + 3, 2064
    x = torch.ones(1, T, D, dtype=torch.bfloat16, device=DEV)
    w = torch.full((D, 4), 0.25, device=DEV)
    y, last = la.short_conv_fwd(x, w, silu=False)
    torch.cuda.synchronize()
    assert bool((y[:, -9:] == 1).all()) and bool((y[:, 0] == 0.25).all()) and bool((last == 1).all())
    dx, dw, _, _ = la.short_conv_bwd(x, w, x, silu=False)
    torch.cuda.synchronize()
    assert bool((dx[:, :5] == 1).all()) and bool((dx[:, -1] == 0.25).all())
    want = torch.tensor([T - 3, T - 2, T - 1, T], dtype=torch.float64, device=DEV)
    # whole numbers below 2^24 add up exactly
    assert bool((dw.double() == want).all())
