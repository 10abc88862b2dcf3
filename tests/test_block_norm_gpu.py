"""block_norm_fwd and _bwd against the rows' norms in fp64 (GPU)."""
import numpy as np
import pytest
import torch

import block_ref as bref
import layer_ref as ref

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = float(np.float32(1e-5))
ALPHA, BETA = float(np.float32(0.7)), 1.5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


# B, T, D, type, residual ("": none), post norm, gate, pre norm, weights, center, sliced rows
CASES = [
    (1, 1, 16, "f32", "f32", True, "row", True, True, False, False),
    (2, 3, 32, "bf16", "bf16", False, "none", True, False, True, True),
    (3, 5, 48, "bf16", "f32", True, "batch", True, True, True, False),
    (1, 7, 256, "f32", "f32", False, "row", False, False, False, True),
    (2, 9, 272, "bf16", "bf16", True, "batch", True, True, False, True),
    (5, 4, 512, "f32", "f32", True, "none", True, True, True, False),
    (1, 33, 528, "bf16", "", True, "row", True, True, False, False),
    (2, 3, 1040, "bf16", "f32", True, "batch", False, True, True, True),
    (3, 70, 2048, "bf16", "bf16", True, "row", True, True, False, False),
    (1, 5, 4096, "f32", "f32", True, "batch", True, True, True, True),
    (2, 3, 4112, "bf16", "bf16", True, "batch", True, True, True, False),
    (1, 400, 8192, "bf16", "f32", True, "row", True, True, True, False),
    (2, 301, 8176, "f32", "f32", False, "batch", True, True, False, True),
    (700, 2, 64, "bf16", "bf16", True, "batch", True, True, False, False),
    (1, 3001, 128, "bf16", "f32", True, "row", True, True, False, False),
    (40, 1, 1024, "bf16", "bf16", False, "row", True, True, False, False),
]
ids = lambda c: "x".join(map(str, c))


def inputs(c, seed=0):
    B, T, D, dt, res, post, gate, pre, weights, center, sliced = c
    g = torch.Generator().manual_seed(seed + B + 7 * T + 11 * D)
    ty, rty = TYPES[dt], TYPES[res or dt]

    def rows(type_, scale):
        t = (torch.randn(B, T, D + (64 if sliced else 0), generator=g) * scale + 0.3).to(type_).to(DEV)
        return t[..., 32:32 + D] if sliced else t

    o, h, dy, dh = rows(ty, 2.0), rows(rty, 3.0) if res else None, rows(ty, 1.0), rows(rty, 1.0)
    vec = lambda: (1 + 0.2 * torch.randn(D, generator=g)).to(DEV)
    wp, wq = (vec() if weights and on else None for on in (post, pre))
    gt = {"none": None, "row": torch.randn(D, generator=g), "batch": torch.randn(B, D, generator=g)}[gate]
    gt = None if gt is None else gt.to(DEV)
    opts = dict(post_norm=post, post_weight=wp, gate=gt, scale=ALPHA, residual_scale=BETA, pre_norm=pre,
                pre_weight=wq, center=center, eps=EPS)
    g64 = None if gt is None else (ref.f64(gt) if gt.dim() == 1 else ref.f64(gt)[:, None])
    plain = dict(post=post, w_post=ref.f64(wp), gate=g64, alpha=ALPHA, beta=BETA, pre=pre, w_pre=ref.f64(wq),
                 center=center, eps=EPS)
    return o, h, dy, dh, opts, plain, rty


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_forward(c):
    o, h, _, _, opts, plain, rty = inputs(c)
    h_new, y = la.block_norm_fwd(o, h, **opts)
    torch.cuda.synchronize()
    want = bref.block(ref.f64(o), ref.f64(h), **plain)
    ref.check("h'", h_new, want[0], want[1], rty)
    assert (y is None) == (not c[7])
    if y is not None:
        ref.check("y", y, want[2], want[3], o.dtype)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_backward(c):
    o, h, dy, dh, opts, plain, rty = inputs(c)
    h_new, _ = la.block_norm_fwd(o, h, **opts)
    dy = dy if c[7] else None
    d_o, d_h, dwp, dg, dwq = la.block_norm_bwd(o, h_new, dy, dh, residual_grad=h is not None, **opts)
    torch.cuda.synchronize()
    want = bref.block_bwd(ref.f64(o), ref.f64(h_new), ref.f64(dy), ref.f64(dh), **plain)
    ref.check("d_o", d_o, *want["o"], o.dtype)
    assert (d_h is None) == (h is None)
    if h is not None:
        ref.check("dh", d_h, *want["h"], rty)
    for name, got, there in (("w_post", dwp, opts["post_weight"]), ("gate", dg, opts["gate"]),
                             ("w_pre", dwq, opts["pre_weight"])):
        assert (got is None) == (there is None)
        if got is not None:
            ref.check(name, got, *want[name], torch.float32)


def test_without_one_of_the_gradients():
    """dh_out None is a zero; without weight_grads and residual_grad the rest is the same."""
    o, h, dy, dh, opts, _, _ = inputs(CASES[2])
    h_new, _ = la.block_norm_fwd(o, h, **opts)
    a = la.block_norm_bwd(o, h_new, dy, None, **opts)
    b = la.block_norm_bwd(o, h_new, dy, torch.zeros_like(dh), **opts)
    c = la.block_norm_bwd(o, h_new, dy, None, weight_grads=False, residual_grad=False, **opts)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(c[0], a[0]) and c[1:] == (None,) * 4


@pytest.mark.parametrize("c", [CASES[3], CASES[8], CASES[11]], ids=ids)
def test_in_place(c):
    o, h, dy, dh, opts, _, _ = inputs(c)
    want, y = la.block_norm_fwd(o, h, **opts)
    dy = dy if c[7] else None
    grads = la.block_norm_bwd(o, want, dy, dh, **opts)
    got, y2 = la.block_norm_fwd(o, h, h_out=h, **opts)
    grads2 = la.block_norm_bwd(o, got, dy, dh, dh=dh, **opts)
    torch.cuda.synchronize()
    assert got is h and torch.equal(h, want) and (y is None or torch.equal(y, y2))
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(grads, grads2))


def test_rows_do_not_touch_each_other():
    """A NaN row stays one, its neighbours keep their bits; what lies beside the rows too."""
    for D in (48, 400, 8192):
        c = (2, 9, D, "bf16", "bf16", True, "row", True, True, True, False)
        o, h, dy, dh, opts, _, _ = inputs(c)
        want = la.block_norm_fwd(o, h, **opts)
        wide = torch.full((2, 9, D + 32), 3.0, dtype=o.dtype, device=DEV)
        bad = o.clone()
        bad[1, 4, 5] = float("nan")
        got = la.block_norm_fwd(bad, h, out=wide[..., 16:16 + D], **opts)
        torch.cuda.synchronize()
        keep = torch.ones(2, 9, dtype=torch.bool, device=DEV)
        keep[1, 4] = False
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(a[1, 4]).all())
        assert bool((wide[..., :16] == 3).all()) and bool((wide[..., 16 + D:] == 3).all())


def test_rows_of_zeros_stay_finite():
    o = torch.zeros(1, 3, 64, device=DEV)
    h, y = la.block_norm_fwd(o, o, post_norm=True, center=True)
    d_o, dh, _, _, _ = la.block_norm_bwd(o, h, torch.ones_like(o), None, post_norm=True, center=True)
    assert bool((y == 0).all()) and bool(torch.isfinite(d_o).all()) and bool(torch.isfinite(dh).all())


def test_no_tokens():
    o, w = torch.zeros(2, 0, 64, device=DEV), torch.ones(64, device=DEV)
    h, y = la.block_norm_fwd(o, o, pre_weight=w, gate=torch.ones(2, 64, device=DEV))
    assert h.shape == y.shape == (2, 0, 64)
    out = la.block_norm_bwd(o, h, y, None, pre_weight=w, gate=torch.ones(2, 64, device=DEV))
    assert bool((out[3] == 0).all()) and out[3].shape == (2, 64) and bool((out[4] == 0).all())


def test_gradients_against_differences():
    c = (2, 5, 96, "f32", "f32", True, "batch", True, True, True, False)
    o, h, dy, dh, opts, plain, _ = inputs(c, seed=3)
    h_new, _ = la.block_norm_fwd(o, h, **opts)
    got = [ref.f64(t) for t in la.block_norm_bwd(o, h_new, dy, dh, **opts)]
    dy, dh = ref.f64(dy), ref.f64(dh)
    at = [ref.f64(o), ref.f64(h), plain["w_post"], plain["gate"][:, 0], plain["w_pre"]]
    rng = np.random.default_rng(1)

    def loss(v):
        p = dict(plain, w_post=v[2], gate=v[3][:, None], w_pre=v[4])
        out = bref.block(v[0], v[1], **p)
        return (out[0] * dh).sum() + (out[2] * dy).sum()

    for i, grad in enumerate(got):
        v = rng.standard_normal(at[i].shape)
        step = lambda s: [a + s * v if j == i else a for j, a in enumerate(at)]
        slope = (loss(step(1e-6)) - loss(step(-1e-6))) / 2e-6
        # fp32 sums of the kernel, and h' rounded to fp32 before the backward pass
        assert abs(slope - (grad * v).sum()) <= 2 ** -16 * np.abs(grad * v).sum() + 1e-5


def test_offsets_past_2_31_elements():
    """Rows of ones: their norm, and the sums over 2^20 rows."""
    T, D = 2 ** 20 + 3, 2064
    o = torch.ones(1, T, D, dtype=torch.bfloat16, device=DEV)
    w = torch.full((D,), 0.5, device=DEV)
    h, y = la.block_norm_fwd(o, o, post_norm=False, scale=3.0, pre_weight=w)
    torch.cuda.synchronize()
    assert bool((h[:, -5:] == 4).all()) and bool((y[:, -5:] == 0.5).all())
    _, dh, _, _, dw = la.block_norm_bwd(o, h, o, None, scale=3.0, pre_weight=w)
    torch.cuda.synchronize()
    # dy n summed over the rows; n = 1 but for eps and roundings
    assert float((dw - T).abs().max()) <= T * 2.0 ** -18
    assert float(dh[:, -5:].abs().max()) <= 2.0 ** -16  # a row of equal entries: its norm does not move
