"""head_gate_fwd and head_gate_bwd against their plain fp64 form (GPU)."""
import numpy as np
import pytest
import torch

import layer_ref as ref

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = float(np.float32(1e-5))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


# B, H, T, d, gate, weight, center, type, layout of o
CASES = [
    (1, 1, 1, 16, True, True, False, "bf16", "heads"),
    (3, 4, 1, 64, True, True, False, "bf16", "heads"),
    (2, 3, 17, 128, True, False, True, "bf16", "heads"),
    (2, 5, 33, 256, True, True, False, "bf16", "rows"),
    (1, 2, 129, 48, False, True, True, "f32", "rows"),
    (2, 2, 21, 240, True, True, True, "f32", "heads"),
    (1, 7, 65, 80, True, True, False, "f32", "padded"),
    (4, 1, 300, 32, False, False, False, "bf16", "padded"),
    (1, 16, 500, 112, True, True, True, "bf16", "heads"),
]


def case(c):
    B, H, T, d, gated, weight, center, dt, layout = c
    g = torch.Generator().manual_seed(sum(c[:4]))
    dt = TYPES[dt]
    o = 3 * torch.randn(B, H, T, d, generator=g) + 0.5
    if layout == "heads":
        o = o.to(dt).to(DEV)
    elif layout == "rows":
        o = o.permute(0, 2, 1, 3).contiguous().to(dt).to(DEV).permute(0, 2, 1, 3)
    else:
        pad = torch.zeros(B, H + 1, T + 3, d + 16).to(dt).to(DEV)
        pad[:, :H, :T, :d] = o.to(dt).to(DEV)
        o = pad[:, :H, :T, :d]
    o[0, 0, 0] = 0 if not center else 2.5  # a row that is all zeros once the mean is out
    gate = (2 * torch.randn(B, T, H, d, generator=g)).to(dt).to(DEV) if gated else None
    if gated:
        gate[0, 0, 0, :4] = torch.tensor([0.0, -200.0, 150.0, torch.finfo(dt).min])
    w = (1 + 0.2 * torch.randn(H, d, generator=g)).to(DEV) if weight else None
    return g, o, gate, w, center


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(map(str, c)))
def test_forward(c):
    _, o, gate, w, center = case(c)
    y = la.head_gate_fwd(o, gate, weight=w, eps=EPS, center=center)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        want, bound = ref.gate(ref.f64(o), ref.f64(gate), ref.f64(w), EPS, center)
    ref.check("y", y, want, bound, y.dtype)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(map(str, c)))
def test_backward(c):
    g, o, gate, w, center = case(c)
    B, H, T, d = o.shape
    dy = torch.randn(B, T, H, d, generator=g).to(o.dtype).to(DEV)
    d_o, dg, dw = la.head_gate_bwd(o, gate, dy, weight=w, eps=EPS, center=center)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        want = ref.gate_bwd(ref.f64(o), ref.f64(gate), ref.f64(dy), ref.f64(w), EPS, center)
    ref.check("d_o", d_o, want[0], want[1], o.dtype)
    assert (dg is None) == (gate is None) and (dw is None) == (w is None)
    if gate is not None:
        ref.check("dgate", dg, want[2], want[3], o.dtype)
    if w is not None:
        ref.check("dweight", dw, want[4], want[5], torch.float32)


def test_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    o = torch.randn(2, 3, 5, 64, generator=g).to(DEV)
    gate, dy = (torch.randn(2, 5, 3, 64, generator=g).to(DEV) for _ in range(2))
    w = (1 + 0.1 * torch.randn(3, 64, generator=g)).to(DEV)
    grads = la.head_gate_bwd(o, gate, dy, weight=w, eps=EPS, center=True)
    at = [ref.f64(t) for t in (o, gate, w)]
    dy = ref.f64(dy)
    rng = np.random.default_rng(0)
    for i, grad in enumerate(grads):
        v = rng.standard_normal(at[i].shape)
        def loss(s):
            a = [x + s * v if j == i else x for j, x in enumerate(at)]
            return (dy * ref.gate(*a, EPS, True)[0]).sum()
        slope = (loss(1e-6) - loss(-1e-6)) / 2e-6
        grad = ref.f64(grad)
        assert abs(slope - (grad * v).sum()) <= 2 ** -18 * np.abs(grad * v).sum() + 1e-5


def test_strided_outputs_leave_what_lies_between():
    g, o, gate, w, center = case(CASES[2])
    w = torch.ones(3, 128, device=DEV)
    B, H, T, d = o.shape
    y = la.head_gate_fwd(o, gate, weight=w, center=center)
    wide = torch.full((B, T + 1, H + 2, d), 5.0, dtype=o.dtype, device=DEV)
    la.head_gate_fwd(o, gate, weight=w, center=center, out=wide[:, :T, 1:1 + H])
    assert torch.equal(wide[:, :T, 1:1 + H], y)
    assert bool((wide[:, T] == 5).all()) and bool((wide[:, :, 0] == 5).all()) and bool((wide[:, :, -1] == 5).all())
    dy = torch.randn(B, T, H, d, generator=g).to(o.dtype).to(DEV)
    want = la.head_gate_bwd(o, gate, dy, weight=w, center=center)
    gw = torch.full((B, T, 2 * H, d), 5.0, dtype=o.dtype, device=DEV)
    ow = torch.full((B, T, 2 * H, d), 5.0, dtype=o.dtype, device=DEV)
    got = la.head_gate_bwd(o, gate, dy, weight=w, center=center, dgate=gw[:, :, H:],
                           d_o=ow[:, :, :H].permute(0, 2, 1, 3))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((gw[:, :, :H] == 5).all()) and bool((ow[:, :, H:] == 5).all())


def test_repeated_gate_and_gradient():
    """A gate shared by all heads (a stride of 0) and a gradient that is the same for
    every token are read like their copies."""
    g = torch.Generator().manual_seed(8)
    o = torch.randn(2, 4, 9, 32, generator=g).to(DEV)
    gate = torch.randn(2, 9, 1, 32, generator=g).to(DEV).expand(2, 9, 4, 32)
    dy = torch.randn(1, 1, 4, 32, generator=g).to(DEV).expand(2, 9, 4, 32)
    assert torch.equal(la.head_gate_fwd(o, gate), la.head_gate_fwd(o, gate.contiguous()))
    got, want = la.head_gate_bwd(o, gate, dy), la.head_gate_bwd(o, gate.contiguous(), dy.contiguous())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens():
    o = torch.zeros(2, 3, 0, 64, device=DEV)
    w = torch.ones(3, 64, device=DEV)
    y = la.head_gate_fwd(o, weight=w)
    assert y.shape == (2, 0, 3, 64)
    assert bool((la.head_gate_bwd(o, None, y, weight=w)[2] == 0).all())


def test_offsets_past_2_31_elements():
    T, H, d = 2 ** 20 + 1, 16, 128
    o = torch.empty(1, H, T, d, dtype=torch.bfloat16, device=DEV).normal_()
    gate = torch.empty(1, T, H, d, dtype=torch.bfloat16, device=DEV).normal_()
    y = la.head_gate_fwd(o, gate)
    torch.cuda.synchronize()
    o_end, g_end = o[:, -2:, -3:], gate[:, -3:, -2:]
    want, bound = ref.gate(ref.f64(o_end), ref.f64(g_end), None, float(np.float32(1e-6)), False)
    ref.check("y", y[:, -3:, -2:], want, bound, torch.bfloat16)
    d_o, dg, _ = la.head_gate_bwd(o, gate, y)
    torch.cuda.synchronize()
    want = ref.gate_bwd(ref.f64(o_end), ref.f64(g_end), ref.f64(y[:, -3:, -2:]), None,
                        float(np.float32(1e-6)), False)
    ref.check("d_o", d_o[:, -2:, -3:], want[0], want[1], torch.bfloat16)
    ref.check("dgate", dg[:, -3:, -2:], want[2], want[3], torch.bfloat16)
