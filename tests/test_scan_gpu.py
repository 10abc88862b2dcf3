"""scan_fwd, scan_bwd and scan_step against the recurrence token by token in fp64 (GPU)."""
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


# B, T, D, type, initial state, restarts
CASES = [
    (1, 1, 16, "f32", True, False),
    (2, 2, 48, "bf16", False, False),
    (3, 7, 64, "f32", True, True),
    (1, 63, 16, "bf16", True, False),
    (1, 64, 32, "f32", False, True),
    (2, 127, 80, "bf16", True, True),
    (1, 128, 208, "f32", True, False),
    (2, 129, 64, "f32", False, False),
    (1, 255, 96, "bf16", True, False),
    (1, 1025, 16, "f32", True, True),
    (3, 1500, 112, "bf16", True, False),
    (1, 5003, 48, "f32", True, True),
    (37, 300, 1024, "bf16", False, True),
    (2, 2049, 192, "f32", True, False),
    (130, 5, 4096, "f32", True, False),
    (160, 130, 48, "bf16", True, True),
    (170, 65, 80, "f32", True, True),
    (3, 700, 3088, "bf16", True, True),
    (2, 5000, 4080, "bf16", True, True),
    (1, 4001, 720, "bf16", True, True),
    (5, 2500, 8208, "bf16", False, False),
    (2, 17, 48, "bf16", True, True),
    (40, 39, 4080, "f32", True, True),
    (33, 64, 4080, "bf16", True, True),
    (7, 16, 80, "bf16", True, True),
]


def inputs(c, seed=0):
    B, T, D, dt, state, restarts = c
    g = torch.Generator().manual_seed(seed + B + 7 * T + 11 * D)
    log_a = -torch.exp(torch.rand(B, T, D, generator=g) * 9.2 - 9.2)
    log_a[torch.rand(B, T, D, generator=g) < 0.01] = 0.0
    log_a[torch.rand(B, T, D, generator=g) < 0.01] = -30.0
    if restarts:
        log_a[torch.rand(B, T, D, generator=g) < 0.02] = float("-inf")
        log_a[torch.rand(B, T, D, generator=g) < 0.01] = -1000.0
    x = torch.randn(B, T, D, generator=g).to(TYPES[dt])
    h0, dT = (torch.randn(B, D, generator=g) if state else None for _ in range(2))
    to = lambda t: None if t is None else t.to(DEV)
    return to(x), to(log_a), to(h0), to(dT), g


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(map(str, c)))
def test_forward(c):
    x, log_a, h0, _, _ = inputs(c)
    h, hT = la.scan_fwd(x, log_a, h0=h0)
    torch.cuda.synchronize()
    want, bound, last, last_bound = ref.scan(ref.f64(x), ref.f64(log_a), ref.f64(h0))
    ref.check("h", h, want, bound, x.dtype)
    ref.check("h_T", hT, last, last_bound, torch.float32)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(map(str, c)))
def test_backward(c):
    x, log_a, h0, dT, g = inputs(c)
    h, _ = la.scan_fwd(x, log_a, h0=h0, return_state=False)
    dh = torch.randn(*x.shape, generator=g).to(x.dtype).to(DEV)
    dx, dla, dh0 = la.scan_bwd(log_a, h, dh, h0=h0, dh_T=dT)
    torch.cuda.synchronize()
    w = ref.scan_bwd(ref.f64(log_a), ref.f64(h), ref.f64(dh), ref.f64(h0), ref.f64(dT))
    ref.check("dx", dx, w[0], w[1], x.dtype)
    ref.check("dlog_a", dla, w[2], w[3], torch.float32)
    ref.check("dh0", dh0, w[4], w[5], torch.float32)


def test_gradients_against_differences():
    x, log_a, h0, dT, g = inputs((2, 40, 32, "f32", True, False), seed=4)
    log_a = log_a.clamp(max=-1e-3)
    h, _ = la.scan_fwd(x, log_a, h0=h0)
    dh = torch.randn(*x.shape, generator=g).to(DEV)
    grads = [ref.f64(t) for t in la.scan_bwd(log_a, h, dh, h0=h0, dh_T=dT)]
    at, dh, dT = [ref.f64(t) for t in (x, log_a, h0)], ref.f64(dh), ref.f64(dT)
    rng = np.random.default_rng(0)
    for i, grad in enumerate(grads):
        v = rng.standard_normal(at[i].shape)
        def loss(s):
            h, _, last, _ = ref.scan(*[a + s * v if j == i else a for j, a in enumerate(at)])
            return (dh * h).sum() + (dT * last).sum()
        slope = (loss(1e-6) - loss(-1e-6)) / 2e-6
        assert abs(slope - (grad * v).sum()) <= 2 ** -18 * np.abs(grad * v).sum() + 1e-5


@pytest.mark.parametrize("T,cut", [(6, 1), (200, 64), (200, 65), (3000, 1999)])
def test_calls_continue_each_other(T, cut):
    """Two calls joined by the state, in place, against one: both within the bounds."""
    x, log_a, h0, _, _ = inputs((2, T, 48, "f32", True, False))
    want, bound, last, last_bound = ref.scan(ref.f64(x), ref.f64(log_a), ref.f64(h0))
    s = h0.clone()
    h1, s1 = la.scan_fwd(x[:, :cut].contiguous(), log_a[:, :cut].contiguous(), h0=s, h_out=s)
    h2, s2 = la.scan_fwd(x[:, cut:].contiguous(), log_a[:, cut:].contiguous(), h0=s, h_out=s)
    torch.cuda.synchronize()
    assert s1 is s and s2 is s
    ref.check("h", torch.cat((h1, h2), 1), want, bound, torch.float32)
    ref.check("h_T", s, last, last_bound, torch.float32)


def test_backward_calls_continue_each_other():
    x, log_a, h0, dT, g = inputs((2, 500, 32, "f32", True, True))
    h, _ = la.scan_fwd(x, log_a, h0=h0)
    dh = torch.randn(2, 500, 32, generator=g).to(DEV)
    w = ref.scan_bwd(ref.f64(log_a), ref.f64(h), ref.f64(dh), ref.f64(h0), ref.f64(dT))
    cut = 177
    part = lambda t, a, b: t[:, a:b].contiguous()
    dx2, dl2, s = la.scan_bwd(part(log_a, cut, 500), part(h, cut, 500), part(dh, cut, 500),
                              h0=h[:, cut - 1].contiguous(), dh_T=dT)
    dx1, dl1, d0 = la.scan_bwd(part(log_a, 0, cut), part(h, 0, cut), part(dh, 0, cut), h0=h0, dh_T=s)
    torch.cuda.synchronize()
    ref.check("dx", torch.cat((dx1, dx2), 1), w[0], w[1], torch.float32)
    ref.check("dlog_a", torch.cat((dl1, dl2), 1), w[2], w[3], torch.float32)
    ref.check("dh0", d0, w[4], w[5], torch.float32)


@pytest.mark.parametrize("T", [40, 700])
def test_nothing_passes_a_restart(T):
    """NaN and infinities before a restart, in x, the state and the gradients, stay
    before it (forward) and behind it (backward)."""
    x, log_a, h0, dT, g = inputs((2, T, 64, "f32", True, False))
    cut = T // 2 + 3
    log_a[:, cut] = float("-inf")
    clean_x, clean_h0 = x.clone(), h0.clone()
    x[:, :cut, ::3], h0[0, ::2] = float("nan"), float("inf")
    h, hT = la.scan_fwd(x, log_a, h0=h0)
    h_c, hT_c = la.scan_fwd(clean_x, log_a, h0=clean_h0)
    torch.cuda.synchronize()
    assert torch.isfinite(hT).all() and torch.equal(h[:, cut:], h_c[:, cut:]) and torch.equal(hT, hT_c)
    assert torch.isnan(h[:, :cut, ::3]).all()
    dh = torch.randn(2, T, 64, generator=g).to(DEV)
    want = la.scan_bwd(log_a, h_c, dh, h0=clean_h0, dh_T=dT)
    bad = dh.clone()
    bad[:, cut:, ::5] = float("nan")
    got = la.scan_bwd(log_a, h_c, bad, h0=clean_h0, dh_T=dT)
    torch.cuda.synchronize()
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a[:, :cut], b[:, :cut])
    assert torch.equal(got[2], want[2])
    # a NaN in the forward's h before the restart reaches no gradient behind it
    got = la.scan_bwd(log_a, h, dh, h0=h0, dh_T=dT)
    torch.cuda.synchronize()
    assert torch.equal(got[1][:, cut:], want[1][:, cut:]) and torch.equal(got[0], want[0])


@pytest.mark.parametrize("B,T,D,dt", [(1, 12, 32, "f32"), (2, 100, 64, "f32"), (2, 100, 48, "bf16"),
                                      (1, 5003, 48, "f32"), (1, 900, 7680, "bf16"),
                                      (3, 700, 3088, "bf16"), (5, 600, 8208, "f32")])
def test_infinities_and_nan_last_until_a_restart(B, T, D, dt):
    """Decays whose product underflows over any run of more than three tokens are no
    restart: what an infinity or a NaN reaches is what the formula says."""
    at, cut = T // 6, T - T // 6
    x = torch.ones(B, T, D, dtype=TYPES[dt], device=DEV)
    log_a = torch.full((B, T, D), -30.0, device=DEV)
    log_a[:, cut] = float("-inf")
    clean, _ = la.scan_fwd(x, log_a)
    bad = x.clone()
    bad[:, at, 0::3], bad[:, at, 1::3] = float("inf"), float("nan")
    h, hT = la.scan_fwd(bad, log_a)
    torch.cuda.synchronize()
    assert bool(torch.isposinf(h[:, at:cut, 0::3]).all()) and bool(torch.isnan(h[:, at:cut, 1::3]).all())
    assert torch.equal(h[:, :at], clean[:, :at]) and torch.equal(h[:, cut:], clean[:, cut:])
    assert torch.equal(h[..., 2::3], clean[..., 2::3]) and bool(torch.isfinite(hT).all())
    # backward: from cut towards the first token, as far as the restart's own dx
    restart = T // 8
    log_a[:, cut], log_a[:, restart] = -30.0, float("-inf")
    want = la.scan_bwd(log_a, clean, x)
    bad = x.clone()
    bad[:, cut, 0::3], bad[:, cut, 1::3] = float("inf"), float("nan")
    dx, dla, dh0 = la.scan_bwd(log_a, clean, bad)
    torch.cuda.synchronize()
    assert bool(torch.isposinf(dx[:, restart:cut + 1, 0::3]).all())
    assert bool(torch.isnan(dx[:, restart:cut + 1, 1::3]).all())
    assert bool(torch.isposinf(dla[:, restart + 1:cut + 1, 0::3]).all())
    for a, b in zip((dx, dla), want):
        assert torch.equal(a[:, :restart], b[:, :restart]) and torch.equal(a[:, cut + 1:], b[:, cut + 1:])
        assert torch.equal(a[..., 2::3], b[..., 2::3])
    assert torch.equal(dh0, want[2])


@pytest.mark.parametrize("B,D,dt", [(1, 16, "f32"), (3, 48, "bf16"), (256, 4096, "bf16"), (5, 1040, "f32")])
def test_step(B, D, dt):
    """One step is a scan of one token, bit for bit; in place or not."""
    x, log_a, h0, _, _ = inputs((B, 1, D, dt, True, True))
    h, hT = la.scan_fwd(x, log_a, h0=h0)
    x1, l1 = x[:, 0].contiguous(), log_a[:, 0].contiguous()
    s = h0.clone()
    new = torch.empty_like(h0)
    out2 = la.scan_step(x1, l1, h0, h_out=new)
    out = la.scan_step(x1, l1, s)
    torch.cuda.synchronize()
    assert torch.equal(out, h[:, 0]) and torch.equal(out2, out)
    assert torch.equal(s, hT) and torch.equal(new, hT)


def test_outputs_end_where_they_end():
    x, log_a, h0, dT, g = inputs((3, 77, 80, "bf16", True, False))
    n = x.numel()
    guard = torch.full((n + 512,), 3.0, dtype=torch.bfloat16, device=DEV)
    want, _ = la.scan_fwd(x, log_a, h0=h0)
    la.scan_fwd(x, log_a, h0=h0, out=guard[256:256 + n].view(x.shape))
    assert torch.equal(guard[256:256 + n].view(x.shape), want)
    assert bool((guard[:256] == 3).all()) and bool((guard[256 + n:] == 3).all())
    wx, wl, _ = la.scan_bwd(log_a, want, x, h0=h0, dh_T=dT)
    fl = torch.full((n + 512,), 3.0, device=DEV)
    la.scan_bwd(log_a, want, x, h0=h0, dh_T=dT, dx=guard[256:256 + n].view(x.shape),
                dlog_a=fl[256:256 + n].view(x.shape))
    torch.cuda.synchronize()
    assert torch.equal(guard[256:256 + n].view(x.shape), wx) and torch.equal(fl[256:256 + n].view(x.shape), wl)
    for t in (guard, fl):
        assert bool((t[:256] == 3).all()) and bool((t[256 + n:] == 3).all())


def test_no_tokens():
    x = torch.zeros(2, 0, 32, device=DEV)
    h0 = torch.randn(2, 32, device=DEV)
    h, hT = la.scan_fwd(x, x, h0=h0)
    assert h.shape == (2, 0, 32) and torch.equal(hT, h0)
    assert bool((la.scan_fwd(x, x)[1] == 0).all())
    assert torch.equal(la.scan_bwd(x, x, x, dh_T=h0)[2], h0)
    assert bool((la.scan_bwd(x, x, x)[2] == 0).all())


def test_offsets_past_2_31_elements():
    """A constant input and decay against the geometric series, past 2^31 elements."""
    T, D, rate = 2 ** 20 + 3, 2064, 2.0 ** -7
    x = torch.ones(1, T, D, dtype=torch.bfloat16, device=DEV)
    log_a = torch.full((1, T, D), -rate, device=DEV)
    h, hT = la.scan_fwd(x, log_a)
    torch.cuda.synchronize()
    full = 1.0 / (1.0 - np.exp(-rate))
    # each of the ~1/rate tokens that count is off by 8 U of the sum: 2^-14 in all
    assert float((hT.double() - full).abs().max()) <= 2.0 ** -14 * full
    assert float((h[:, -5:].double() - full).abs().max()) <= (2.0 ** -8 + 2.0 ** -14) * full
    dx, dla, dh0 = la.scan_bwd(log_a, h, x)
    torch.cuda.synchronize()
    assert float((dx[:, :5].double() - full).abs().max()) <= (2.0 ** -8 + 2.0 ** -14) * full
    assert float((dx[:, -1].double() - 1).abs().max()) <= 2.0 ** -8
    c = np.exp(-rate) * full
    assert float((dh0.double() - c).abs().max()) <= 2.0 ** -13 * c
    want = np.exp(-rate) * h[:, -2].double()  # the last token: c = a dh
    assert float(((dla[:, -1].double() - want).abs() / want).max()) <= 2.0 ** -20


def test_a_wait_that_runs_out_is_reported(opts):
    """The cluster's exchange, muted: both walks return after their limit of 1 ms with
    the status set, and the next calls are whole again."""
    x, log_a, h0, _, _ = inputs((1, 5003, 48, "f32", True, True))
    want, _ = la.scan_fwd(x, log_a, h0=h0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for call in (lambda: la.scan_fwd(x, log_a, h0=h0, dev_status=status),
                 lambda: la.scan_bwd(log_a, want, x, h0=h0, dev_status=status)):
        opts.force_timeout()
        status.zero_()
        call()
        torch.cuda.synchronize()
        assert int(status) == la.LA_ERR_TIMEOUT
        opts.force_timeout(False)
        status.zero_()
        call()
        got, _ = la.scan_fwd(x, log_a, h0=h0, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == 0 and torch.equal(got, want)
