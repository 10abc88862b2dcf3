"""ssm_fwd, ssm_bwd and ssm_step against the recurrence token by token in fp64 (GPU)."""
import numpy as np
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


# B, T, D, N, G, type, gate, skip, bias, softplus, state, positions, sliced
CASES = [
    (1, 1, 16, 16, 1, "f32", True, True, True, True, True, False, False),
    (2, 1, 48, 8, 2, "bf16", False, False, False, False, False, False, True),
    (1, 2, 16, 64, 1, "f32", False, True, True, True, True, True, False),
    (3, 7, 80, 32, 1, "f32", True, False, True, True, False, True, True),
    (2, 8, 208, 16, 2, "bf16", True, True, True, True, True, False, False),
    (1, 9, 32, 64, 2, "f32", False, True, False, False, True, True, True),
    (2, 31, 144, 8, 1, "f32", True, True, True, True, True, True, False),
    (1, 33, 272, 16, 1, "f32", True, True, True, True, True, True, True),
    (2, 65, 112, 32, 2, "f32", True, True, False, True, False, False, False),
    (1, 100, 64, 64, 1, "bf16", True, True, True, True, True, True, True),
    (3, 257, 48, 16, 3, "f32", True, True, True, True, True, True, False),
    (1, 300, 128, 16, 1, "f32", False, False, False, False, True, False, False),
    (2, 500, 16, 8, 1, "bf16", True, True, True, True, True, True, False),
    (1, 1025, 32, 16, 2, "f32", True, False, True, True, True, True, False),
    (1, 777, 16, 32, 1, "f32", True, True, True, True, False, True, True),
    (1, 521, 16, 64, 1, "f32", False, True, True, False, True, False, False),
    (9, 40, 528, 16, 1, "bf16", True, True, True, True, True, False, True),
    (64, 3, 1040, 8, 5, "f32", True, True, True, True, True, False, False),
    (16, 5, 1552, 16, 1, "bf16", True, True, True, True, True, True, False),
    (24, 4, 2048, 8, 1, "f32", True, True, True, True, True, True, False),
    (24, 3, 2064, 16, 2, "f32", False, True, True, True, True, False, False),
    (10, 4, 2048, 32, 1, "f32", True, True, True, True, True, False, False),
    (20, 2, 1040, 64, 1, "f32", True, True, True, True, True, True, False),
]
ids = lambda c: "x".join(map(str, c))


def inputs(c, seed=0):
    B, T, D, N, G, dt, gate, skip, bias, softplus, state, positions, sliced = c
    g = torch.Generator().manual_seed(seed + B + 7 * T + 11 * D + 13 * N)
    ty = TYPES[dt]
    to = lambda t: t.to(DEV)

    def rows(width, scale=1.0):
        t = to((torch.randn(B, T, width + (48 if sliced else 0), generator=g) * scale).to(ty))
        return t[..., 16:16 + width] if sliced else t

    x, z, dy = rows(D), rows(D), rows(D)
    usual = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)
    if softplus:
        step = rows(D, 2.0)
    else:
        step = to((usual * (0.5 + torch.rand(B, T, D, generator=g))).to(ty))
    b, c_ = (rows(G * N).unflatten(-1, (G, N)) for _ in range(2))
    A = to(-(torch.arange(1, N + 1) * (0.5 + torch.rand(D, N, generator=g))))
    A[:, 0] = 0.0  # a state that does not decay
    s = dict(x=x, dt=step, A=A, b=b, c=c_)
    opts = dict(skip=to(torch.randn(D, generator=g)) if skip else None, gate=z if gate else None,
                dt_bias=to(torch.log(torch.expm1(usual)) if softplus else usual) if bias else None, softplus=softplus,
                h0=to(torch.randn(B, D, N, generator=g)) if state else None, positions=None)
    if positions:
        opts["positions"] = to((torch.rand(B, T, generator=g) > 0.05).to(torch.int32) * 3)
    dh_T = to(torch.randn(B, D, N, generator=g)) if state else None
    return s, opts, dy, dh_T


def plain(s, opts):
    v = {n: None if t is None else ref.f64(t) for n, t in {**s, **opts}.items() if n not in ("softplus", "positions")}
    pos = None if opts["positions"] is None else opts["positions"].cpu().numpy()
    return (v["x"], v["dt"], v["A"], v["b"], v["c"], v["skip"], v["gate"], v["dt_bias"], opts["softplus"], v["h0"], pos)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_forward(c):
    s, opts, _, _ = inputs(c)
    y, hT = la.ssm_fwd(**s, **opts)
    torch.cuda.synchronize()
    want, bound, last, last_bound = bref.ssm(*plain(s, opts))
    ref.check("h_T", hT, last, last_bound, torch.float32)
    ref.check("y", y, want, bound, y.dtype)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_backward(c):
    s, opts, dy, dh_T = inputs(c)
    out = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    want = bref.ssm_bwd(*plain(s, opts), ref.f64(dy), ref.f64(dh_T))
    ty = s["x"].dtype
    for name, got, dtype in zip(("x", "dt", "A", "b", "c", "skip", "gate", "bias", "h0"), out,
                                (ty, ty, torch.float32, ty, ty, torch.float32, ty, torch.float32, torch.float32)):
        assert (got is None) == (name not in want), name
        if got is not None:
            ref.check("d" + name, got, *want[name], dtype)


def test_gradients_against_differences():
    c = (2, 40, 32, 8, 2, "f32", True, True, True, True, True, False, False)
    s, opts, dy, dh_T = inputs(c, seed=4)
    got = [ref.f64(t) for t in la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)]
    at = list(plain(s, opts))
    dy, dh_T = ref.f64(dy), ref.f64(dh_T)
    where = [0, 1, 2, 3, 4, 5, 6, 7, 9]  # x, dt, A, b, c, skip, gate, bias, h0
    rng = np.random.default_rng(0)
    for grad, k in zip(got, where):
        v = rng.standard_normal(at[k].shape)

        def loss(step):
            y, _, last, _ = bref.ssm(*[a + step * v if i == k else a for i, a in enumerate(at)])
            return (y * dy).sum() + (last * dh_T).sum()

        slope = (loss(1e-6) - loss(-1e-6)) / 2e-6
        assert abs(slope - (grad * v).sum()) <= 2 ** -16 * np.abs(grad * v).sum() + 1e-5


@pytest.mark.parametrize("T,cut", [(6, 1), (200, 64), (700, 333)])
def test_calls_continue_each_other(T, cut):
    """Two calls joined by the state, in place, against one: both within the bounds."""
    c = (2, T, 48, 16, 1, "f32", True, True, True, True, True, True, False)
    s, opts, dy, dh_T = inputs(c)
    want, bound, last, last_bound = bref.ssm(*plain(s, opts))
    h = opts["h0"].clone()
    ys = []
    for a, b in ((0, cut), (cut, T)):
        part = {n: t if n == "A" else t[:, a:b] for n, t in s.items()}
        o = dict(opts, h0=h, gate=opts["gate"][:, a:b], positions=opts["positions"][:, a:b].contiguous())
        y, same = la.ssm_fwd(**part, **o, h_out=h)
        assert same is h
        ys.append(y)
    torch.cuda.synchronize()
    ref.check("y", torch.cat(ys, 1), want, bound, torch.float32)
    ref.check("h_T", h, last, last_bound, torch.float32)


@pytest.mark.parametrize("T", [40, 700])
def test_nothing_passes_a_document(T):
    """NaN and infinities before a document's start reach nothing behind it, forward, nor
    before it, backward."""
    c = (2, T, 64, 16, 1, "f32", True, True, True, True, True, False, False)
    s, opts, dy, dh_T = inputs(c)
    cut = T // 2 + 3
    opts["positions"] = torch.ones(2, T, dtype=torch.int32, device=DEV)
    opts["positions"][:, cut] = 0
    y, hT = la.ssm_fwd(**s, **opts)
    want = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    bad = dict(s, x=s["x"].clone(), b=s["b"].clone())
    bad["x"][:, :cut, ::3], bad["b"][:, :cut, :, ::5] = float("nan"), float("inf")
    h0 = opts["h0"].clone()
    h0[:, ::2] = float("inf")
    y2, hT2 = la.ssm_fwd(**bad, **dict(opts, h0=h0))
    got = la.ssm_bwd(*s.values(), torch.where(torch.arange(T, device=DEV)[:, None] >= cut, float("nan"), dy), dh_T=dh_T,
                     **opts)
    back = la.ssm_bwd(*bad.values(), dy, dh_T=dh_T, **dict(opts, h0=h0))
    torch.cuda.synchronize()
    assert torch.equal(y[:, cut:], y2[:, cut:]) and torch.equal(hT, hT2) and bool(torch.isfinite(hT).all())
    for i in (0, 1, 3, 4, 6):
        assert torch.equal(got[i][:, :cut], want[i][:, :cut])
        assert torch.equal(back[i][:, cut:], want[i][:, cut:])
    assert torch.equal(got[8], want[8])


@pytest.mark.parametrize("B,D,N,G,dt,sliced", [(1, 16, 8, 1, "f32", False), (3, 48, 16, 2, "bf16", True),
                                               (256, 2048, 16, 1, "bf16", False), (5, 1040, 32, 1, "f32", True),
                                               (7, 80, 64, 1, "f32", False)])
def test_step(B, D, N, G, dt, sliced):
    c = (B, 1, D, N, G, dt, True, True, True, True, True, False, sliced)
    s, opts, _, _ = inputs(c)
    one = {n: t if n == "A" else t[:, 0] for n, t in s.items()}
    o = {n: opts[n] for n in ("skip", "dt_bias", "softplus")}
    o["gate"] = opts["gate"][:, 0]
    new = torch.empty_like(opts["h0"])
    y = la.ssm_step(**one, h=opts["h0"], h_out=new, **o)
    h = opts["h0"].clone()
    y2 = la.ssm_step(**one, h=h, **o)
    torch.cuda.synchronize()
    want, bound, last, last_bound = bref.ssm(*plain(s, opts))
    ref.check("y", y.unsqueeze(1), want, bound, y.dtype)
    ref.check("h", new, last, last_bound, torch.float32)
    assert torch.equal(y, y2) and torch.equal(h, new)


def test_outputs_end_where_they_end():
    c = (3, 77, 80, 16, 1, "bf16", True, True, True, True, True, False, False)
    s, opts, dy, dh_T = inputs(c)
    B, T, D = s["x"].shape
    want, _ = la.ssm_fwd(**s, **opts)
    wide = torch.full((B, T, 3 * D), 3.0, dtype=want.dtype, device=DEV)
    la.ssm_fwd(**s, **opts, out=wide[..., D:2 * D])
    grads = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    gw = torch.full((B, T, 3 * D + 64), 3.0, dtype=want.dtype, device=DEV)  # dx, ddt, dgate, db, dc side by side
    at = [gw[..., :D], gw[..., D:2 * D], gw[..., 2 * D:3 * D], gw[..., 3 * D + 16:3 * D + 32], gw[..., 3 * D + 32:3 * D + 48]]
    got = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts, dx=at[0], ddt=at[1], dgate=at[2], db=at[3].unsqueeze(2),
                     dc=at[4].unsqueeze(2))
    torch.cuda.synchronize()
    assert torch.equal(wide[..., D:2 * D], want)
    assert bool((wide[..., :D] == 3).all()) and bool((wide[..., 2 * D:] == 3).all())
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    assert bool((gw[..., 3 * D:3 * D + 16] == 3).all()) and bool((gw[..., 3 * D + 48:] == 3).all())


def test_a_cut_sequence_needs_its_workspace():
    """Long sequences of few channels are cut: without room for the chunks' states the call
    is refused (on the host, its pointers untouched)."""
    import ctypes
    lib, at = la.library(), lambda k: 0x10000000 + 0x100000 * k
    need = lib.la_ssm_workspace_size(1, 4096, 16, 8, 1, 1)
    assert need > 0

    def call(ws, size):
        return lib.la_ssm_fwd(at(0), at(1), at(2), at(3), at(4), None, None, None, None, 1, 1, 4096, 16, 8, 1, 1, None,
                              None, at(9), None, ws, size, None)

    for ws, size in ((None, 0), (at(11) + 4, need), (at(11), need - 1), (at(9), need), (at(3), need)):
        assert call(ws, ctypes.c_size_t(size)) == la.LA_ERR_INVALID_ARG
    x = torch.zeros(1, 4096, 16, device=DEV)
    with pytest.raises(ValueError, match="workspace"):
        la.ssm_fwd(x, x, torch.zeros(16, 8, device=DEV), x[..., :8], x[..., 8:],
                   workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_no_tokens():
    x, A = torch.zeros(2, 0, 32, device=DEV), torch.ones(32, 8, device=DEV)
    b, h0 = torch.zeros(2, 0, 8, device=DEV), torch.randn(2, 32, 8, device=DEV)
    y, h = la.ssm_fwd(x, x, A, b, b, h0=h0)
    assert y.shape == (2, 0, 32) and torch.equal(h, h0)
    assert bool((la.ssm_fwd(x, x, A, b, b)[1] == 0).all())
    out = la.ssm_bwd(x, x, A, b, b, x, dh_T=h0, skip=A[:, 0].contiguous())
    assert bool((out[2] == 0).all()) and bool((out[5] == 0).all()) and torch.equal(out[8], h0)


def test_steps_of_any_size():
    """softplus from far below to far above: its relative error holds for tiny steps too."""
    v = torch.cat((torch.linspace(-85, 90, 3999), torch.tensor([0.0])))
    D, T = 16, 250
    dt = v.view(1, T, D).to(DEV)
    x, A = torch.ones(1, T, D, device=DEV), torch.zeros(D, 8, device=DEV)
    b = torch.zeros(1, T, 8, device=DEV)
    b[..., 0] = 1.0
    pos = torch.zeros(1, T, dtype=torch.int32, device=DEV)  # every token alone: y = delta
    for ty, extra in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        y, _ = la.ssm_fwd(x.to(ty), dt.to(ty), A, b.to(ty), b.to(ty), positions=pos)
        torch.cuda.synchronize()
        want = np.logaddexp(ref.f64(dt.to(ty)), 0.0)
        rel = (16 + 4 * np.abs(ref.f64(dt.to(ty)))) * ref.U + 4 * ref.U + extra
        assert (np.abs(ref.f64(y) - want) <= rel * want + 1e-37).all()


def test_a_step_of_zero_leaves_the_state():
    """delta = 0 and rates of 0: the state's bits stay as they are, for thousands of tokens."""
    T, D = 3001, 48
    x, b = torch.ones(1, T, D, device=DEV), torch.ones(1, T, 16, device=DEV)
    h0 = torch.randn(1, D, 16, generator=torch.Generator().manual_seed(3)).to(DEV)
    A = -torch.rand(D, 16, device=DEV)
    _, h = la.ssm_fwd(x, torch.zeros_like(x), A, b, b, softplus=False, h0=h0)
    dh0 = la.ssm_bwd(x, torch.zeros_like(x), A, b, torch.zeros_like(b), x, softplus=False, h0=h0, dh_T=h0)[8]
    step = h0.clone()
    la.ssm_step(x[:, 0], torch.zeros(1, D, device=DEV), A, b[:, 0], b[:, 0], step, softplus=False)
    _, still = la.ssm_fwd(torch.zeros_like(x), x, torch.zeros_like(A), b, b, softplus=False, h0=h0)
    torch.cuda.synchronize()
    assert torch.equal(h, h0) and torch.equal(dh0, h0) and torch.equal(step, h0) and torch.equal(still, h0)


def test_slow_decays_do_not_drift():
    """One impulse carried through 4000 tokens at each decay: its size is e^(sum) within the mean error a
    decay may have (1e-8 of itself, and the exponent's own rounding)."""
    T, D, N = 4000, 16, 8
    A = -torch.logspace(-1, 0.5, D * N, base=10.0).view(D, N).to(DEV)
    dt = torch.full((1, T, D), 0.02, device=DEV)
    x, b = torch.zeros(1, T, D, device=DEV), torch.ones(1, T, N, device=DEV)
    h0 = torch.ones(1, D, N, device=DEV)
    _, h = la.ssm_fwd(x, dt, A, b, b, softplus=False, h0=h0)
    torch.cuda.synchronize()
    want = np.exp(T * float(np.float32(0.02)) * ref.f64(A))
    size = T * 0.02 * np.abs(ref.f64(A))
    keep = want > 1e-30
    rel = np.abs(ref.f64(h)[0] - want) / want
    # a token's decay: 1e-8 on average and 2^-24 of its argument, twice; a product's rounding, random
    assert (rel <= T * 1.2e-8 + 2 * size * 2.0 ** -24 + 8 * T ** 0.5 * 2.0 ** -24)[keep].all()


def test_results_repeat():
    c = (3, 257, 48, 16, 3, "f32", True, True, True, True, True, True, False)
    s, opts, dy, dh_T = inputs(c)
    a = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    b = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_past_2_31_elements():
    """A constant input and decay against the geometric series, past 2^31 elements."""
    T, D, N = 2 ** 20 + 3, 2064, 8
    x = torch.ones(1, T, D, dtype=torch.bfloat16, device=DEV)
    A = torch.full((D, N), -1.0, device=DEV)
    A[:, 1] = -2.0
    b = torch.zeros(1, T, N, dtype=torch.bfloat16, device=DEV)
    b[..., 0], b[..., 1] = 1.0, 1.0
    step = 2.0 ** -7
    dt = x * step
    y, h = la.ssm_fwd(x, dt, A, b, b, softplus=False)
    torch.cuda.synchronize()
    full = [step / (1 - np.exp(-k * step)) for k in (1, 2)]
    # each of the ~1/step tokens that count is off by 16 U of the sum: 2^-13 in all
    for n in (0, 1):
        assert float((h[:, :, n].double() - full[n]).abs().max()) <= 2.0 ** -13 * full[n]
    assert float((y[:, -5:].double() - sum(full)).abs().max()) <= (2.0 ** -8 + 2.0 ** -13) * sum(full)
