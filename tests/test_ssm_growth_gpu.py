"""Decays above 1 (A above 0, or steps below 0 without softplus) through a sequence cut into
chunks (GPU): a state of zero stays zero and a small one grows, as token by token, although
the decay over a whole chunk passes the fp32 range."""
import itertools

import pytest
import torch

import block_ref as bref
import layer_ref as ref
from test_ssm_gpu import plain

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


def sequence(T, D, N, sign, step):
    """Inputs of one sequence whose even channels grow by e^step a token (at most) and whose odd
    ones decay; with sign -1 both delta and A are below 0."""
    g = torch.Generator().manual_seed(T + N)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)
    grows = (torch.arange(D, device=DEV) % 2 == 0)[:, None]
    rate = 0.5 + 0.5 * torch.rand(D, N, generator=g).to(DEV)
    # delta is `sign * step` everywhere: A of its sign grows, of the other decays
    A = sign * torch.where(grows, rate, -rate)
    dt = torch.full((1, T, D), sign * step, device=DEV)
    return dict(x=r(1, T, D), dt=dt, A=A, b=r(1, T, N), c=r(1, T, N)), r(1, T, D), grows[:, 0]


def check(s, opts, dy, dh_T):
    """Outputs and gradients, entry by entry, against the walk token by token in fp64."""
    y, hT = la.ssm_fwd(**s, **opts)
    grads = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    four = dict(s, b=s["b"].unsqueeze(2), c=s["c"].unsqueeze(2))
    p = plain(four, opts)
    want, bound, last, last_bound = bref.ssm(*p)
    ref.check("y", y, want, bound, y.dtype)
    ref.check("h_T", hT, last, last_bound, torch.float32)
    v = bref.ssm_bwd(*p, ref.f64(dy), ref.f64(dh_T))
    for name, got in zip(("x", "dt", "A", "b", "c", "skip", "gate", "bias", "h0"), grads):
        if got is not None:
            (w, e), shape = v[name], ref.f64(got).shape
            ref.check("d" + name, got, w.reshape(shape), e.reshape(shape), got.dtype)


def options(**over):
    return {**dict(skip=None, gate=None, dt_bias=None, softplus=False, h0=None, positions=None), **over}


@pytest.mark.parametrize("N,sign,start", list(itertools.product([8, 16, 64], [1, -1], [False, True])))
def test_a_state_of_zero_does_not_grow(N, sign, start):
    """e^4 a token over chunks of 32 tokens and more: x is 0 in the growing channels but for the
    last three tokens, dy but for the first three."""
    T, D = 1000, 32
    s, dy, grows = sequence(T, D, N, sign, 4.0)
    s["x"][:, :T - 3, grows] = 0.0
    dy[:, 3:, grows] = 0.0
    pos = None
    if start:
        pos = torch.ones(1, T, dtype=torch.int32, device=DEV)
        pos[0, 333] = pos[0, 700] = 0
    check(s, options(positions=pos), dy, None)


def test_a_state_of_zero_does_not_grow_behind_softplus():
    T, D, N = 700, 32, 16
    s, dy, grows = sequence(T, D, N, 1, 4.0)
    s["x"][:, :T - 3, grows] = 0.0
    dy[:, 3:, grows] = 0.0
    h0 = torch.where(grows[:, None], 0.0, 1.0).expand(D, N)[None].contiguous()
    check(s, options(softplus=True, h0=h0), dy, torch.zeros_like(h0))


@pytest.mark.parametrize("sign", [1, -1])
def test_a_small_state_grows_and_a_small_gradient(sign):
    """1e-30 times e^88 and more, within one chunk's first 48 tokens: the decay alone is past the range,
    its product with the state (and with the gradient behind) is not."""
    T, D, N = 600, 32, 16
    s, dy, grows = sequence(T, D, N, sign, 2.0)
    s["A"] = sign * torch.where(grows[:, None], 1.0, -0.25).expand(D, N).contiguous()
    s["dt"][:, 48:] = 0.0
    s["x"][:, :, grows] = 0.0
    dy[:, :, grows] = 0.0
    dy[:, 50, grows] = 1e-30
    h0 = torch.where(grows[:, None], 1e-30, 1.0).expand(D, N)[None].contiguous()
    check(s, options(h0=h0), dy, torch.zeros_like(h0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,at,start", [(300, 150, None), (300, 150, 200), (300, 150, 120), (700, 640, 660), (700, 600, 660),
                                        (5000, 2500, None), (5000, 2500, 2600)])
def test_a_step_that_is_not_a_number_stays_so(T, at, start, dtype):
    """A NaN step: its channel's states behind it and gradients before it are NaN up to a document's
    start, where no gradient comes in behind it too; the other channels keep their bits."""
    D, N, ch = 32, 16, 5
    s, dy, _ = sequence(T, D, N, 1, 0.01)
    s["A"] = -s["A"].abs()
    dy[:, at - 10:, ch] = 0.0
    s, dy = {n: t if n == "A" else t.to(dtype) for n, t in s.items()}, dy.to(dtype)
    pos = None
    if start is not None:
        pos = torch.ones(1, T, dtype=torch.int32, device=DEV)
        pos[0, start] = 0
    h0 = torch.ones(1, D, N, device=DEV)
    opts, grad = options(h0=h0, positions=pos), options(h0=h0, positions=pos, dh_T=torch.zeros_like(h0))
    y, hT = la.ssm_fwd(**s, **opts)
    want = la.ssm_bwd(*s.values(), dy, **grad)
    s["dt"] = s["dt"].clone()
    s["dt"][0, at, ch] = float("nan")
    y2, hT2 = la.ssm_fwd(**s, **opts)
    got = la.ssm_bwd(*s.values(), dy, **grad)
    torch.cuda.synchronize()
    others = [k for k in range(D) if k != ch]
    end = T if start is None or start < at else start
    begin = 0 if start is None or start > at else start  # gradients pass back to here
    nan = torch.isnan(y2[0, :, ch])
    assert bool(nan[at:end].all()) and not bool(nan[:at].any()) and not bool(nan[end:].any())
    assert torch.equal(y2[..., others], y[..., others]) and torch.equal(hT2[:, others], hT[:, others])
    assert bool(torch.isnan(hT2[0, ch]).all()) == (end == T)
    dx, ddt, dh0 = got[0], got[1], got[8]
    for v, w in ((dx, want[0]), (ddt, want[1])):
        nan = torch.isnan(v[0, :, ch])
        assert bool(nan[begin:at + 1].all()) and not bool(nan[:begin].any())
        assert torch.equal(v[..., others], w[..., others])
    assert bool(torch.isnan(dh0[0, ch]).all()) == (begin == 0)
    assert torch.equal(dh0[:, others], want[8][:, others])
