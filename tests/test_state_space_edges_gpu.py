"""The state space operators at the edges (GPU): every shape of the walks, documents at the
borders of tiles, blocks and chunks, repeated rows, two calls at once, infinities that must
not spread."""
import numpy as np
import pytest
import torch

import block_ref as bref
import layer_ref as ref
from test_ssm_gpu import inputs, plain

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


def check_all(s, opts, dy, dh_T, y, hT, grads):
    p = plain(s, opts)
    want, bound, last, last_bound = bref.ssm(*p)
    ref.check("y", y, want, bound, y.dtype)
    ref.check("h_T", hT, last, last_bound, torch.float32)
    v = bref.ssm_bwd(*p, ref.f64(dy), ref.f64(dh_T))
    for name, got in zip(("x", "dt", "A", "b", "c", "skip", "gate", "bias", "h0"), grads):
        if got is not None:
            ref.check("d" + name, got, *v[name], got.dtype)


# the walks with sixteen states a lane (many channels) and with four, cut into chunks or not,
# in bf16 and fp32, with a last tile of channels that is not full
@pytest.mark.parametrize("c", [(24, 20, 2048, 8, 1, "bf16", True, True, True, True, True, True, False),
                               (10, 19, 2064, 32, 1, "bf16", True, True, True, True, True, True, True),
                               (20, 17, 1040, 64, 1, "bf16", True, True, True, True, True, False, False),
                               (2, 700, 272, 16, 1, "bf16", True, True, True, True, True, True, False),
                               (2, 705, 272, 16, 1, "f32", True, True, True, True, True, True, True),
                               (2, 700, 48, 8, 1, "f32", True, True, True, True, True, True, False),
                               (1, 600, 80, 32, 2, "bf16", True, False, True, True, True, True, False)],
                         ids=lambda c: "x".join(map(str, c)))
def test_every_walk(c):
    s, opts, dy, dh_T = inputs(c)
    y, hT = la.ssm_fwd(**s, **opts)
    grads = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    check_all(s, opts, dy, dh_T, y, hT, grads)


@pytest.mark.parametrize("at", [0, 7, 8, 15, 16, 31, 32, 63, 64, 127, 128, 639])
def test_a_document_that_starts_anywhere(at):
    c = (1, 640, 32, 16, 1, "f32", True, True, True, True, True, False, False)
    s, opts, dy, dh_T = inputs(c)
    opts["positions"] = torch.full((1, 640), 5, dtype=torch.int32, device=DEV)
    opts["positions"][0, at] = 0
    y, hT = la.ssm_fwd(**s, **opts)
    grads = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    check_all(s, opts, dy, dh_T, y, hT, grads)


@pytest.mark.parametrize("T", [7, 8, 9, 15, 16, 17, 24, 33, 511, 512, 513])
def test_lengths_around_the_tiles(T):
    c = (2, T, 48, 16, 1, "bf16", True, True, True, True, True, False, False)
    s, opts, dy, dh_T = inputs(c)
    y, hT = la.ssm_fwd(**s, **opts)
    grads = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    check_all(s, opts, dy, dh_T, y, hT, grads)


def test_every_token_a_document():
    """No state passes anywhere: y is each token's own, the gradients too."""
    c = (2, 300, 32, 16, 1, "f32", True, True, True, True, True, False, False)
    s, opts, dy, dh_T = inputs(c)
    opts["positions"] = torch.zeros(2, 300, dtype=torch.int32, device=DEV)
    opts["h0"].fill_(float("nan"))
    y, hT = la.ssm_fwd(**s, **opts)
    grads = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    opts["h0"] = None
    check_all(s, opts, dy, dh_T, y, hT, grads[:8] + (None,))
    assert bool((grads[8] == 0).all())
    pos = opts["positions"]
    x, w = s["x"], torch.randn(32, 4, generator=torch.Generator().manual_seed(1)).to(DEV)
    y, _ = la.short_conv_fwd(x, w, silu=False, state=torch.full((2, 3, 32), float("inf"), device=DEV), positions=pos)
    assert torch.equal(y, x * w[:, 3])


def test_rows_repeated_by_a_stride_of_zero():
    """One sequence's rows read for every batch entry: the same as a copy for each."""
    B, T, D, N = 3, 40, 64, 16
    g = torch.Generator().manual_seed(5)
    one = [torch.randn(1, T, w, generator=g).bfloat16().to(DEV) for w in (D, D, N, N, D)]
    A = -torch.rand(D, N, generator=g).to(DEV)
    wide = [t.expand(B, T, -1) for t in one]
    full = [t.contiguous() for t in wide]
    h0 = torch.randn(B, D, N, generator=g).to(DEV)
    outs = [la.ssm_fwd(v[0], v[1], A, v[2], v[3], gate=v[4], h0=h0) for v in (wide, full)]
    grads = [la.ssm_bwd(v[0], v[1], A, v[2], v[3], full[0], gate=v[4], h0=h0) for v in (wide, full)]
    w = torch.randn(D, 3, generator=g).to(DEV)
    conv = [la.short_conv_fwd(v[0], w) for v in (wide, full)]
    back = [la.short_conv_bwd(v[0], w, v[4]) for v in (wide, full)]
    block = [la.block_norm_fwd(v[0], v[1], post_norm=True) for v in (wide, full)]
    bb = [la.block_norm_bwd(v[0], block[1][0], v[4], None, post_norm=True) for v in (wide, full)]
    torch.cuda.synchronize()
    for pair in (outs, grads, conv, back, block, bb):
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(*pair))
    with pytest.raises(la.LinAttnError):  # rows of an output may not lie on each other
        la.ssm_fwd(full[0], full[1], A, full[2], full[3], out=torch.empty_like(one[0]).expand(B, T, D))
    with pytest.raises(la.LinAttnError):
        la.short_conv_fwd(full[0], w, out=torch.empty_like(one[0]).expand(B, T, D))
    with pytest.raises(la.LinAttnError):
        la.block_norm_fwd(full[0], one[1].expand(B, T, D), h_out=one[1].expand(B, T, D))


def test_calls_at_once_on_two_streams():
    c = (2, 900, 48, 16, 1, "f32", True, True, True, True, True, True, False)
    sets = [inputs(c, seed=k) for k in (1, 2)]
    want = [(la.ssm_fwd(**s, **o), la.ssm_bwd(*s.values(), dy, dh_T=d, **o)) for s, o, dy, d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for (s, o, dy, d), st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append((la.ssm_fwd(**s, **o), la.ssm_bwd(*s.values(), dy, dh_T=d, **o)))
        torch.cuda.synchronize()
        for (f, b), (wf, wb) in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(f + b, wf + wb))


def test_a_workspace_given_and_more_than_needed():
    c = (1, 900, 32, 16, 1, "bf16", True, True, True, True, True, True, False)
    s, opts, dy, dh_T = inputs(c)
    want, grads = la.ssm_fwd(**s, **opts), la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    room = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever it is read unwritten
    got = la.ssm_fwd(**s, **opts, workspace=room)
    room.fill_(255)
    back = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts, workspace=room)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + back, want + grads))
    x, w = s["x"], torch.ones(32, 4, device=DEV)
    a = la.short_conv_bwd(x, w, dy)
    room.fill_(255)
    b = la.short_conv_bwd(x, w, dy, workspace=room)
    p = torch.ones(32, device=DEV)
    u = la.block_norm_bwd(x, x, dy, None, pre_weight=p, gate=torch.ones(1, 32, device=DEV))
    room.fill_(255)
    v = la.block_norm_bwd(x, x, dy, None, pre_weight=p, gate=torch.ones(1, 32, device=DEV), workspace=room)
    torch.cuda.synchronize()
    assert all(m is None and n is None or torch.equal(m, n) for m, n in zip(a + u, b + v))


def test_positions_anywhere_in_a_buffer():
    c = (1, 50, 32, 16, 1, "f32", True, True, True, True, True, True, False)
    s, opts, dy, dh_T = inputs(c)
    for shift in (1, 2, 3):
        buf = torch.zeros(64, dtype=torch.int32, device=DEV)
        buf[shift:shift + 50] = opts["positions"][0]
        moved = dict(opts, positions=buf[shift:shift + 50].view(1, 50))
        w = torch.ones(32, 4, device=DEV)
        for f in (lambda o: la.ssm_fwd(**s, **o), lambda o: la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **o),
                  lambda o: la.short_conv_fwd(s["x"], w, positions=o["positions"]),
                  lambda o: la.short_conv_bwd(s["x"], w, dy, positions=o["positions"])):
            assert all(a is None or torch.equal(a, b) for a, b in zip(f(opts), f(moved)))


def test_a_residual_in_fp32_without_one_before_it():
    o = torch.randn(2, 5, 96, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    h = torch.empty(2, 5, 96, device=DEV)
    got, y = la.block_norm_fwd(o, None, h_out=h, scale=2.0)
    torch.cuda.synchronize()
    assert got is h and torch.equal(h, 2.0 * o.float())
    want = bref.block(ref.f64(o), None, False, None, None, 2.0, 1.0, True, None, False, float(np.float32(1e-6)))
    ref.check("y", y, want[2], want[3], o.dtype)


def test_steps_and_reads_in_one_graph():
    """A captured decode step replayed: the states move on in place each time."""
    B, D, N = 3, 64, 16
    g = torch.Generator().manual_seed(8)
    x = torch.randn(B, D, generator=g).bfloat16().to(DEV)
    b, A = torch.randn(B, N, generator=g).bfloat16().to(DEV), -torch.rand(D, N, generator=g).to(DEV)
    w = torch.randn(D, 4, generator=g).to(DEV)
    cs, h = torch.zeros(B, 3, D, dtype=torch.bfloat16, device=DEV), torch.zeros(B, D, N, device=DEV)

    def step():
        u = la.short_conv_step(x, w, cs)
        y = la.ssm_step(u, u, A, b, b, h)
        return la.block_norm_fwd(y[:, None], None)[1]

    step()
    cs.zero_(), h.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    cs.zero_(), h.zero_()
    want = [step().clone() for _ in range(4)]
    end = (cs.clone(), h.clone())
    cs.zero_(), h.zero_()
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])
    assert torch.equal(cs, end[0]) and torch.equal(h, end[1])


@pytest.mark.parametrize("D", [48, 512, 528, 2048, 4096, 8192])
@pytest.mark.parametrize("dtypes", [("f32", "f32"), ("bf16", "f32")], ids="-".join)
def test_rows_at_any_multiple_of_16_bytes(D, dtypes):
    """Rows of every width that begin 16 bytes behind a multiple of 32 give what dense ones give."""
    B, T = 2, 5
    to, th = ({"f32": torch.float32, "bf16": torch.bfloat16}[d] for d in dtypes)
    g = torch.Generator().manual_seed(D)
    dense = [torch.randn(B, T, D, generator=g).to(t).to(DEV) for t in (to, th, to, th)]
    pre, post, gate = (torch.randn(D, generator=g).to(DEV) for _ in range(3))
    opts = dict(post_norm=True, post_weight=post, pre_weight=pre, gate=gate, scale=0.5, residual_scale=0.75, center=True)

    def moved(t):
        e = 16 // t.element_size()
        buf = torch.zeros(B, T, D + 2 * e + e, dtype=t.dtype, device=DEV)
        return buf[:, :, e:e + D]

    def run(place):
        o, h, dy, dh = (place(t).copy_(t) for t in dense)
        h_out, y, d_o, d_h = (place(t) for t in (h, o, o, h))
        la.block_norm_fwd(o, h, h_out=h_out, out=y, **opts)
        grads = la.block_norm_bwd(o, h_out, dy, dh, d_o=d_o, dh=d_h, **opts)
        return h_out, y, *grads

    want, got = run(torch.empty_like), run(moved)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    f64 = [ref.f64(t) for t in dense]
    p = bref.block(f64[0], f64[1], True, ref.f64(post), ref.f64(gate), 0.5, 0.75, True, ref.f64(pre), True,
                   float(np.float32(1e-6)))
    ref.check("h'", got[0], p[0], p[1], th)
    ref.check("y", got[1], p[2], p[3], to)


def test_a_decay_of_zero_drops_nothing():
    """An infinite state times a decay that underflows is not a number, in a sequence cut into
    chunks (T at least 512) as in two calls that are not; a document's start drops it in both."""
    B, T, D, N = 1, 1000, 32, 16
    g = torch.Generator().manual_seed(3)
    x, b = torch.randn(B, T, D, generator=g).to(DEV), torch.randn(B, T, N, generator=g).to(DEV)
    dt, A = torch.full((B, T, D), 40.0, device=DEV), torch.full((D, N), -50.0, device=DEV)
    h0 = torch.zeros(B, D, N, device=DEV)
    h0[0, 3] = float("inf")
    dh = torch.zeros(B, D, N, device=DEV)
    dh[0, 5] = float("inf")
    for start in (None, 700):
        pos = None
        if start is not None:
            pos = torch.ones(B, T, dtype=torch.int32, device=DEV)
            pos[0, start] = 0
        cut = lambda t, lo, hi: None if t is None else t[:, lo:hi].contiguous()
        y, hT = la.ssm_fwd(x, dt, A, b, b, h0=h0, positions=pos)
        parts, h = [], h0
        for lo, hi in ((0, 400), (400, T - 200), (T - 200, T)):
            p, h = la.ssm_fwd(*(cut(t, lo, hi) for t in (x, dt)), A, *(cut(t, lo, hi) for t in (b, b)), h0=h,
                              positions=cut(pos, lo, hi))
            parts.append(p)
        dh0 = la.ssm_bwd(x, dt, A, b, b, torch.zeros_like(x), h0=torch.zeros_like(h0), positions=pos, dh_T=dh)[8]
        torch.cuda.synchronize()
        whole = torch.cat(parts, 1)
        assert torch.equal(torch.isnan(y), torch.isnan(whole)) and torch.equal(torch.isnan(hT), torch.isnan(h))
        there = torch.isnan(y)[0].any(0)
        assert bool(there[3]) and int(there.sum()) == 1
        assert bool(torch.isnan(y[0, -1, 3])) == (start is None)
        assert bool(torch.isnan(dh0[0, 5]).all()) == (start is None) and not bool(torch.isnan(dh0[0, 4]).any())
