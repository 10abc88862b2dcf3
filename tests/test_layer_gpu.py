"""The operators around retention used together (GPU): a retention mixer forward,
backward and token by token, the recurrence with its norm and gate, streams and
captured graphs."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import oracle
import pins

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
TOL = 2e-2  # retention itself in bf16: its own tolerance, of the largest entry
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


def close(name, got, want, tol=TOL):
    err = pins.rel_err(ref.f64(got), want)
    assert err <= tol, f"{name}: {err:.3e}"


def mixer_inputs(B=2, T=150, H=4, d=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    packed = torch.randn(B, T, 3 * H, d, generator=g).bfloat16().to(DEV)
    gate = torch.randn(B, T, H, d, generator=g).bfloat16().to(DEV)
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).to(DEV) for _ in range(2))
    w = (1 + 0.1 * torch.randn(H, d, generator=g)).to(DEV)
    return packed, gate, wq, wk, w, [1 - 2.0 ** (-5 - h) for h in range(H)]


def mixer(packed, gate, wq, wk, w, gamma, H, **where):
    opts = dict(interleaved=True, q_weight=wq, k_weight=wk, k_scale=0.125)
    q, k = la.qk_rotate_fwd(packed[:, :, :H], packed[:, :, H:2 * H], **opts, **where)
    v = packed[:, :, 2 * H:].transpose(1, 2).contiguous()
    o, S, _ = la.chunk_fwd(q, k, v, gamma)
    return la.head_gate_fwd(o, gate, weight=w), q, k, v, o, S


def test_mixer_forward_and_backward():
    B, T, H, d = 2, 150, 4, 64
    packed, gate, wq, wk, w, gamma = mixer_inputs()
    y, q, k, v, o, _ = mixer(packed, gate, wq, wk, w, gamma, H)
    dy = torch.randn(B, T, H, d, generator=torch.Generator().manual_seed(9)).bfloat16().to(DEV)
    d_o, dgate, dw = la.head_gate_bwd(o, gate, dy, weight=w)
    dqr, dkr, dv, _, _ = la.chunk_bwd(q, k, v, d_o, gamma)
    dpacked = torch.zeros_like(packed)
    _, _, dwq, dwk = la.qk_rotate_bwd(packed[:, :, :H], packed[:, :, H:2 * H], dqr, dkr, interleaved=True,
                                      q_weight=wq, k_weight=wk, k_scale=0.125, dq=dpacked[:, :, :H],
                                      dk=dpacked[:, :, H:2 * H])
    torch.cuda.synchronize()
    # link by link in fp64: every operator on the very tensors the one before it handed
    # over (its rounding to bf16 belongs to the hand-over; behind a norm it is not small:
    # token 0 has o = (q.k) v, and dO, perpendicular to o, leaves dq = (dO.v) k = 0 but
    # for roundings)
    x = ref.f64(packed)
    pos = np.broadcast_to(np.arange(T), (B, T))
    r = dict(pos=pos, rot=d, freq=np.array(la.rotary_frequencies(d)), interleaved=True, norm=True, eps=EPS)
    for got, ww, h, s in ((q, wq, 0, 1.0), (k, wk, H, 0.125)):
        ref.check("q, k", got, *ref.qk(x[:, :, h:h + H], w=ref.f64(ww), scale=s, **r), got.dtype)
    O, _, _ = oracle.recurrent(q, k, v, gamma)
    close("o", o, O)
    g64, w64 = ref.f64(gate), ref.f64(w)
    ref.check("y", y, *ref.gate(ref.f64(o), g64, w64, EPS, False), y.dtype)
    want = ref.gate_bwd(ref.f64(o), g64, ref.f64(dy), w64, EPS, False)
    ref.check("d_o", d_o, want[0], want[1], d_o.dtype)
    ref.check("dgate", dgate, want[2], want[3], dgate.dtype)
    ref.check("dw", dw, want[4], want[5], torch.float32)
    dQ, dK, dV, _, _ = oracle.recurrent_bwd(q, k, v, gamma, d_o)
    for name, a, b in (("dq", dqr, dQ), ("dk", dkr, dK), ("dv", dv, dV)):
        close(name, a, b)
    for got, dyr, ww, h, s in ((dwq, dqr, wq, 0, 1.0), (dwk, dkr, wk, H, 0.125)):
        dx, bound, dwx, dwb = ref.qk_bwd(x[:, :, h:h + H], ref.f64(dyr), w=ref.f64(ww), scale=s, **r)
        ref.check("dq, dk", dpacked[:, :, h:h + H], dx, bound, dpacked.dtype)
        ref.check("dq_weight, dk_weight", got, dwx, dwb, torch.float32)
    assert bool((dpacked[:, :, 2 * H:] == 0).all())


def test_decoding_continues_the_prefill():
    """Tokens one at a time (T = 1, a position per sequence, recurrent_step, the gate)
    against the prefill of the whole: q and k bit for bit, o within retention's
    tolerance of the oracle's, y the gate of that o."""
    B, T, H, d, head = 2, 40, 4, 64, 30
    packed, gate, wq, wk, w, gamma = mixer_inputs(T=T, seed=2)
    _, q_all, k_all, v_all, _, _ = mixer(packed, gate, wq, wk, w, gamma, H)
    _, _, _, _, _, S = mixer(packed[:, :head], gate[:, :head], wq, wk, w, gamma, H)
    os_ = []
    for t in range(head, T):
        row = packed[:, t:t + 1]
        q, k = la.qk_rotate_fwd(row[:, :, :H], row[:, :, H:2 * H], interleaved=True, q_weight=wq, k_weight=wk,
                                k_scale=0.125, positions=torch.full((B, 1), t, dtype=torch.int32, device=DEV))
        assert torch.equal(q[:, :, 0], q_all[:, :, t]) and torch.equal(k[:, :, 0], k_all[:, :, t])
        o = la.recurrent_step(q[:, :, 0], k[:, :, 0], row[:, 0, 2 * H:].contiguous(), gamma, S)
        y = la.head_gate_fwd(o[:, :, None], gate[:, t:t + 1], weight=w)
        torch.cuda.synchronize()
        ref.check(f"token {t}", y, *ref.gate(ref.f64(o)[:, :, None], ref.f64(gate[:, t:t + 1]), ref.f64(w),
                                             EPS, False), y.dtype)
        os_.append(o)
    O, _, _ = oracle.recurrent(q_all, k_all, v_all, gamma)
    close("o", torch.stack(os_, 2), O[:, :, head:])


def test_recurrence_with_norm_and_gate():
    """scan -> head_gate and back: the recurrence's rows are read as heads by strides,
    and its gradient comes back in the rows' layout."""
    B, T, H, d = 2, 200, 3, 64
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, T, H * d, generator=g).to(DEV)
    log_a = -torch.rand(B, T, H * d, generator=g).to(DEV)
    gate, dy = (torch.randn(B, T, H, d, generator=g).to(DEV) for _ in range(2))
    h, _ = la.scan_fwd(x, log_a)
    as_heads = h.view(B, T, H, d).permute(0, 2, 1, 3)
    y = la.head_gate_fwd(as_heads, gate, center=True)
    d_h, dgate, _ = la.head_gate_bwd(as_heads, gate, dy, center=True)
    dh = d_h.permute(0, 2, 1, 3).reshape(B, T, H * d)
    assert dh.data_ptr() == d_h.data_ptr()  # no copy: the gradient has the rows' order
    dx, dla, _ = la.scan_bwd(log_a, h, dh)
    torch.cuda.synchronize()
    f32 = torch.float32
    ref.check("h", h, *ref.scan(ref.f64(x), ref.f64(log_a), None)[:2], f32)
    ref.check("y", y, *ref.gate(ref.f64(as_heads), ref.f64(gate), None, EPS, True), f32)
    want = ref.gate_bwd(ref.f64(as_heads), ref.f64(gate), ref.f64(dy), None, EPS, True)
    ref.check("d_h", d_h, want[0], want[1], f32)
    ref.check("dgate", dgate, want[2], want[3], f32)
    want = ref.scan_bwd(ref.f64(log_a), ref.f64(h), ref.f64(dh), None, None)
    ref.check("dx", dx, want[0], want[1], f32)
    ref.check("dlog_a", dla, want[2], want[3], f32)


def all_calls(t, stream=None):
    """Every entry point once on the tensors of t; returns all outputs."""
    kw = dict(stream=stream)
    q, k = la.qk_rotate_fwd(t["q"], t["q"], q_weight=t["w1"], k_weight=t["w1"], **kw)
    gr = la.qk_rotate_bwd(t["q"], t["q"], q, k, q_weight=t["w1"], k_weight=t["w1"], **kw)
    y = la.head_gate_fwd(q, t["q"], weight=t["w2"], **kw)
    gg = la.head_gate_bwd(q, t["q"], y, weight=t["w2"], **kw)
    h, hT = la.scan_fwd(t["x"], t["log_a"], h0=t["h0"], **kw)
    gs = la.scan_bwd(t["log_a"], h, t["x"], h0=t["h0"], dh_T=hT, **kw)
    new = torch.empty_like(hT)
    o = la.scan_step(t["x"][:, 0].contiguous(), t["log_a"][:, 0].contiguous(), hT, h_out=new, **kw)
    return [q, k, *gr, y, *gg, h, hT, *gs, o, new]


def tensors(seed, B=2, T=130, H=3, d=64):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)
    return dict(q=r(B, T, H, d).bfloat16(), w1=1 + 0.1 * r(d), w2=1 + 0.1 * r(H, d),
                x=r(B, T, 96).bfloat16(), log_a=-r(B, T, 96).abs(), h0=r(B, 96))


@pytest.mark.parametrize("how", ["argument", "handle", "current"])
def test_on_another_stream(how):
    """A side stream, given or current: the work and what it allocates belong to it."""
    t = tensors(1)
    want = all_calls(t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            if how == "current":
                got = all_calls(t)
        if how == "argument":
            with torch.cuda.stream(side):
                x1, l1 = t["x"][:, 0].contiguous(), t["log_a"][:, 0].contiguous()
            q, k = la.qk_rotate_fwd(t["q"], t["q"], q_weight=t["w1"], k_weight=t["w1"], stream=side)
            gr = la.qk_rotate_bwd(t["q"], t["q"], q, k, q_weight=t["w1"], k_weight=t["w1"], stream=side)
            y = la.head_gate_fwd(q, t["q"], weight=t["w2"], stream=side)
            gg = la.head_gate_bwd(q, t["q"], y, weight=t["w2"], stream=side)
            h, hT = la.scan_fwd(t["x"], t["log_a"], h0=t["h0"], stream=side)
            gs = la.scan_bwd(t["log_a"], h, t["x"], h0=t["h0"], dh_T=hT, stream=side)
            new = torch.empty_like(hT)
            torch.cuda.current_stream().wait_stream(side)
            side.wait_stream(torch.cuda.current_stream())
            o = la.scan_step(x1, l1, hT, h_out=new, stream=side)
            got = [q, k, *gr, y, *gg, h, hT, *gs, o, new]
        if how == "handle":
            q, k = la.qk_rotate_fwd(t["q"], t["q"], q_weight=t["w1"], k_weight=t["w1"],
                                    stream=side.cuda_stream)
            y = la.head_gate_fwd(q, t["q"], weight=t["w2"], stream=side.cuda_stream)
            h, hT = la.scan_fwd(t["x"], t["log_a"], h0=t["h0"], stream=side.cuda_stream)
            side.synchronize()
            assert torch.equal(q, want[0]) and torch.equal(y, want[6])
            assert torch.equal(h, want[10]) and torch.equal(hT, want[11])
            continue
        side.synchronize()
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))


def test_results_repeat_bit_for_bit():
    t = tensors(2, B=3, T=700, H=5)
    first = all_calls(t)
    for _ in range(3):
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(all_calls(t), first))


def test_two_captured_graphs_replay_side_by_side():
    """Two graphs of every call, each with the memory of its own capture, replayed at
    the same time on two streams with inputs written after the capture."""
    graphs, outs, ts = [], [], []
    pool = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        t = tensors(10 + i)
        with torch.cuda.stream(pool[i]):
            all_calls(t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=pool[i]):
            outs.append(all_calls(t))
        graphs.append(g)
        ts.append(t)
    fresh = [tensors(20 + i) for i in range(2)]
    for t, f in zip(ts, fresh):
        for n in t:
            t[n].copy_(f[n])
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, pool):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, f in zip(outs, fresh):
        want = all_calls(f)
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(out, want))


def test_refuses_a_short_workspace_and_a_wrong_device():
    t = tensors(3)
    q, k = la.qk_rotate_fwd(t["q"], t["q"])
    with pytest.raises(ValueError):
        la.qk_rotate_bwd(t["q"], t["q"], q, k, q_weight=t["w1"],
                         workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        la.head_gate_fwd(q, t["q"].cpu())
    with pytest.raises(ValueError):
        la.scan_fwd(t["x"], t["log_a"].cpu())
    with pytest.raises(la.LinAttnError) as e:  # a row that starts off a 16-byte boundary
        big = torch.zeros(2, 5, 3, 72, dtype=torch.bfloat16, device=DEV)
        la.qk_rotate_fwd(big[..., 4:68], big[..., 4:68])
    assert e.value.status == la.LA_ERR_INVALID_ARG
    with pytest.raises(la.LinAttnError):  # in place: refused
        la.scan_fwd(t["x"], t["log_a"], out=t["x"])
    torch.cuda.synchronize()
