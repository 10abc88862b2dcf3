"""qk_rotate_fwd and qk_rotate_bwd against their plain fp64 form (GPU)."""
import numpy as np
import pytest
import torch

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


def heads(g, layout, B, T, H, d, dt, extra=2):
    """[B,T,H,d] values: dense, a slice of a packed row, the layout [B,H,T,d], or one
    token repeated by a stride of 0."""
    if layout == "packed":
        return torch.randn(B, T, H + extra, d, generator=g).to(dt).to(DEV)[:, :, 1:1 + H]
    if layout == "heads":
        return torch.randn(B, H, T, d, generator=g).to(dt).to(DEV).permute(0, 2, 1, 3)
    if layout == "repeat":
        return torch.randn(B, 1, H, d, generator=g).to(dt).to(DEV).expand(B, T, H, d)
    return torch.randn(B, T, H, d, generator=g).to(dt).to(DEV)


# B, T, Hq, Hk, d, rot, interleaved, norm, weight, type, layout, positions
CASES = [
    (1, 1, 1, 1, 16, 16, True, True, True, "bf16", "dense", None),
    (2, 1, 3, 3, 64, 64, True, True, True, "bf16", "packed", "each"),
    (3, 5, 4, 2, 128, 128, True, True, True, "bf16", "packed", None),
    (2, 37, 8, 8, 128, 128, False, True, True, "bf16", "packed", "each"),
    (2, 19, 5, 1, 80, 32, False, True, False, "f32", "dense", "each"),
    (1, 130, 2, 7, 96, 96, True, True, True, "f32", "heads", 4000),
    (2, 33, 3, 3, 256, 256, False, True, True, "bf16", "heads", None),
    (1, 257, 2, 2, 240, 16, True, True, False, "bf16", "dense", 17),
    (2, 9, 2, 2, 48, 0, True, True, True, "f32", "packed", None),
    (1, 12, 6, 3, 32, 32, False, False, False, "bf16", "repeat", None),
    (4, 300, 16, 4, 64, 48, False, True, True, "f32", "packed", "each"),
    (1, 6, 33, 1, 176, 96, True, False, False, "f32", "packed", "far"),
    (2, 4, 2, 2, 128, 128, False, True, True, "bf16", "dense", "far"),
]


def case(c):
    B, T, Hq, Hk, d, rot, inter, norm, weight, dt, layout, posn = c
    g = torch.Generator().manual_seed(sum(c[:6]) + 13 * inter)
    dt = TYPES[dt]
    q, k = heads(g, layout, B, T, Hq, d, dt), heads(g, layout, B, T, Hk, d, dt)
    if B * T * Hq > 2:
        q = q.clone() if layout == "repeat" else q
        q[-1, -1, 0] = 0  # a row of zeros stays one
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(DEV) if weight else None for _ in range(2))
    pos = np.broadcast_to(np.arange(T), (B, T))
    opts = dict(rot=rot, interleaved=inter, norm=norm, q_weight=wq, k_weight=wk, eps=1e-5, q_scale=0.25,
                k_scale=-1.5)
    if posn == "each":
        pos = torch.randint(-100, 70000, (B, T), generator=g, dtype=torch.int32)
    elif posn == "far":
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, T), generator=g, dtype=torch.int32)
        pos[0, 0], pos[-1, -1] = 2 ** 31 - 1, -2 ** 31
    elif posn is not None:
        opts["pos0"] = posn
        pos = pos + posn
    if torch.is_tensor(pos):
        opts["positions"] = pos.to(DEV)
        pos = pos.numpy()
    freq = la.rotary_frequencies(rot)
    if rot == 96:  # other frequencies than the default ones, a negative one among them
        freq = [f * 0.37 for f in freq]
        freq[1] = -0.9
        opts["inv_freq"] = np.array(freq)
    r = dict(pos=pos, rot=rot, freq=np.array(freq), interleaved=inter, norm=norm, eps=float(np.float32(1e-5)))
    return g, q, k, wq, wk, opts, r


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(map(str, c)))
def test_forward(c):
    _, q, k, wq, wk, opts, r = case(c)
    yq, yk = la.qk_rotate_fwd(q, k, **opts)
    torch.cuda.synchronize()
    for y, x, w, s, name in ((yq, q, wq, 0.25, "q"), (yk, k, wk, -1.5, "k")):
        want, bound = ref.qk(ref.f64(x), w=ref.f64(w), scale=s, **r)
        ref.check(name, y, want, bound, y.dtype)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(map(str, c)))
def test_backward(c):
    g, q, k, wq, wk, opts, r = case(c)
    B, T, Hq, d = q.shape
    Hk = k.shape[2]
    gq = torch.randn(B, Hq, T, d, generator=g).to(q.dtype).to(DEV)
    gk = torch.randn(B, Hk, T, d, generator=g).to(q.dtype).to(DEV)
    dq, dk, dwq, dwk = la.qk_rotate_bwd(q, k, gq, gk, **opts)
    torch.cuda.synchronize()
    assert (dwq is None) == (wq is None)
    for dx, dw, x, dy, w, s, name in ((dq, dwq, q, gq, wq, 0.25, "q"), (dk, dwk, k, gk, wk, -1.5, "k")):
        want, bound, want_w, bound_w = ref.qk_bwd(ref.f64(x), ref.f64(dy), w=ref.f64(w), scale=s, **r)
        ref.check("d" + name, dx, want, bound, dx.dtype)
        if w is not None:
            ref.check(f"d{name}_weight", dw, want_w, bound_w, torch.float32)


def test_gradients_against_differences():
    """A directional derivative of the fp64 form by central differences."""
    c = (2, 7, 3, 2, 64, 64, False, True, True, "f32", "packed", None)
    g, q, k, wq, wk, opts, r = case(c)
    gq = torch.randn(2, 3, 7, 64, generator=g).to(DEV)
    gk = torch.randn(2, 2, 7, 64, generator=g).to(DEV)
    dq, _, dwq, _ = la.qk_rotate_bwd(q, k, gq, gk, **opts)
    x, dy, w = ref.f64(q), ref.f64(gq), ref.f64(wq)
    loss = lambda x, w: (dy * ref.qk(x, w=w, scale=0.25, **r)[0]).sum()
    rng = np.random.default_rng(0)
    # the zero row's curvature is 1 / eps: its direction is left out
    for at, grad, f in ((x, ref.f64(dq), lambda v: loss(v, w)), (w, ref.f64(dwq), lambda v: loss(x, v))):
        v = rng.standard_normal(at.shape)
        if at is x:
            v[-1, -1, 0] = 0
        slope = (f(at + 1e-6 * v) - f(at - 1e-6 * v)) / 2e-6
        # fp32 gradients: their bound, 2^-18 of each term, and the difference's own error
        assert abs(slope - (grad * v).sum()) <= 2 ** -18 * np.abs(grad * v).sum() + 1e-5


def test_weights_on_one_side_and_no_weight_gradients():
    g, q, k, wq, _, opts, r = case(CASES[3])
    opts["k_weight"] = None
    gq = torch.randn(2, 8, 37, 128, generator=g).to(q.dtype).to(DEV)
    dq, dk, dwq, dwk = la.qk_rotate_bwd(q, k, gq, gq, **opts)
    dq2, dk2, none, none2 = la.qk_rotate_bwd(q, k, gq, gq, weight_grads=False, **opts)
    assert dwk is None and none is None and none2 is None
    assert torch.equal(dq, dq2) and torch.equal(dk, dk2)
    want, bound, want_w, bound_w = ref.qk_bwd(ref.f64(q), ref.f64(gq), w=ref.f64(wq), scale=0.25, **r)
    ref.check("dq_weight", dwq, want_w, bound_w, torch.float32)
    want, bound, _, _ = ref.qk_bwd(ref.f64(k), ref.f64(gq), w=None, scale=-1.5, **r)
    ref.check("dk", dk, want, bound, dk.dtype)


def test_gradients_into_a_packed_row_leave_the_rest():
    """dq and dk as slices of one gradient row: the entries between and behind them
    keep what they held."""
    g, q, k, _, _, opts, _ = case((3, 11, 4, 2, 64, 64, True, True, True, "bf16", "packed", None))
    gq = torch.randn(3, 4, 11, 64, generator=g).bfloat16().to(DEV)
    gk = torch.randn(3, 2, 11, 64, generator=g).bfloat16().to(DEV)
    plain = la.qk_rotate_bwd(q, k, gq, gk, **opts)
    row = torch.full((3, 12, 9, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    dq, dk = row[:, :11, 1:5], row[:, :11, 6:8]
    out = la.qk_rotate_bwd(q, k, gq, gk, dq=dq, dk=dk, **opts)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, plain))
    rest = torch.ones(9, dtype=torch.bool)
    rest[1:5] = rest[6:8] = False
    assert bool((row[:, :, rest.to(DEV)] == 7).all()) and bool((row[:, 11] == 7).all())


def test_outputs_end_where_they_end():
    _, q, k, _, _, opts, _ = case(CASES[4])
    B, T, Hq, d = q.shape
    n = B * T * Hq * d
    guard = torch.full((n + 512,), 3.0, device=DEV)
    want, _ = la.qk_rotate_fwd(q, k, **opts)
    la.qk_rotate_fwd(q, k, q_out=guard[256:256 + n].view(B, Hq, T, d), **opts)
    torch.cuda.synchronize()
    assert torch.equal(guard[256:256 + n].view(B, Hq, T, d), want)
    assert bool((guard[:256] == 3).all()) and bool((guard[256 + n:] == 3).all())


def test_positions_and_pos0_agree_with_a_longer_call():
    """Tokens 5.. on their own are those tokens of the whole call, bit for bit."""
    g = torch.Generator().manual_seed(5)
    q = torch.randn(2, 40, 3, 64, generator=g).bfloat16().to(DEV)
    whole = la.qk_rotate_fwd(q, q)[0]
    tail = la.qk_rotate_fwd(q[:, 5:], q[:, 5:], pos0=5)[0]
    one = la.qk_rotate_fwd(q[:, 9:10], q[:, 9:10],
                           positions=torch.full((2, 1), 9, dtype=torch.int32, device=DEV))[0]
    assert torch.equal(whole[:, :, 5:], tail) and torch.equal(whole[:, :, 9:10], one)


def test_no_tokens():
    w = torch.ones(64, device=DEV)
    q = torch.zeros(2, 0, 3, 64, device=DEV)
    yq, yk = la.qk_rotate_fwd(q, q)
    assert yq.shape == (2, 3, 0, 64)
    out = la.qk_rotate_bwd(q, q, yq, yk, q_weight=w, k_weight=w)
    assert out[0].shape == q.shape and bool((out[2] == 0).all()) and bool((out[3] == 0).all())


def test_offsets_past_2_31_elements():
    T, H, d = 2 ** 20 + 1, 16, 128
    q = torch.empty(1, T, H, d, dtype=torch.bfloat16, device=DEV).normal_()
    k = q[:, :, :1]
    yq, yk = la.qk_rotate_fwd(q, k)
    torch.cuda.synchronize()
    last = q[:, -3:, -2:]
    want, bound = ref.qk(ref.f64(last), np.arange(T - 3, T)[None], d, np.array(la.rotary_frequencies(d)),
                         False, True, None, float(np.float32(1e-6)), 1.0)
    ref.check("q", yq[:, -2:, -3:], want, bound, torch.bfloat16)
    dq, dk, _, _ = la.qk_rotate_bwd(q, k, yq, yk)
    torch.cuda.synchronize()
    want, bound, _, _ = ref.qk_bwd(ref.f64(last), ref.f64(yq[:, -2:, -3:]), np.arange(T - 3, T)[None], d,
                                   np.array(la.rotary_frequencies(d)), False, True, None,
                                   float(np.float32(1e-6)), 1.0)
    ref.check("dq", dq[:, -3:, -2:], want, bound, torch.bfloat16)
