"""short_conv, ssm and block_norm used together (GPU): a state space block in its residual
stream forward, backward and token by token, on other streams and from captured graphs."""
import numpy as np
import pytest
import torch

import block_ref as bref
import layer_ref as ref

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


class Block:
    """h -> norm -> (x, gate) -> convolution -> scan -> norm, gate row and residual."""

    def __init__(self, D=64, E=96, N=16, dtype=torch.float32, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(DEV)
        self.D, self.E, self.N, self.ty = D, E, N, dtype
        self.w_in, self.w_bc = r(D, 2 * E, scale=D ** -0.5).to(dtype), r(E, E + 2 * N, scale=E ** -0.5).to(dtype)
        self.w_out = r(E, D, scale=E ** -0.5).to(dtype)
        self.w_pre, self.w_post, self.gate = 1 + r(D, scale=0.1), 1 + r(D, scale=0.1), r(D)
        self.conv_w, self.conv_b = r(E, 4, scale=0.5), r(E)
        self.A = -torch.arange(1, N + 1, device=DEV) * (0.5 + torch.rand(E, N, generator=g).to(DEV))
        self.skip, self.bias = r(E), r(E) - 4.0

    def seam(self):
        return dict(post_norm=True, post_weight=self.w_post, gate=self.gate, pre_weight=self.w_pre, eps=EPS)

    def inner(self, y, conv_state=None, h0=None, positions=None, **where):
        """The block on normed rows y: its output and what the next token needs."""
        E, N = self.E, self.N
        xz = y @ self.w_in
        x, cs = la.short_conv_fwd(xz[..., :E], self.conv_w, bias=self.conv_b, state=conv_state, positions=positions,
                                  **where)
        p = x @ self.w_bc
        u, h = la.ssm_fwd(x, p[..., :E], self.A, p[..., E:E + N], p[..., E + N:], skip=self.skip, gate=xz[..., E:],
                          dt_bias=self.bias, h0=h0, positions=positions, **where)
        return (xz, x, p, u), u @ self.w_out, cs, h

    def step(self, y, cs, h):
        E, N = self.E, self.N
        xz = y @ self.w_in
        x = la.short_conv_step(xz[:, :E], self.conv_w, cs, bias=self.conv_b)
        p = x @ self.w_bc
        u = la.ssm_step(x, p[:, :E], self.A, p[:, E:E + N], p[:, E + N:], h, skip=self.skip, gate=xz[:, E:],
                        dt_bias=self.bias)
        return u @ self.w_out


def stream(B, T, D, dtype=torch.float32, seed=1):
    return torch.randn(B, T, D, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def forward(m, h):
    _, y = la.block_norm_fwd(h, None, pre_weight=m.w_pre, eps=EPS)
    parts, o, cs, s = m.inner(y)
    h1, y1 = la.block_norm_fwd(o, h, **m.seam())
    return y, parts, o, cs, s, h1, y1


def test_block_forward_link_by_link():
    """Each operator on the very tensors the one before it handed over."""
    m, (B, T) = Block(), (2, 150)
    h = stream(B, T, m.D)
    y, (xz, x, p, u), o, cs, s, h1, y1 = forward(m, h)
    torch.cuda.synchronize()
    E, N = m.E, m.N
    f = ref.f64
    first = bref.block(f(h), None, False, None, None, 1.0, 1.0, True, f(m.w_pre), False, EPS)
    ref.check("y", y, first[2], first[3], m.ty)
    want = bref.conv(f(xz[..., :E]), f(m.conv_w), f(m.conv_b), True, None, None)
    ref.check("x", x, want[0], want[1], m.ty)
    four = lambda t: f(t).reshape(B, T, 1, N)
    want = bref.ssm(f(x), f(p[..., :E]), f(m.A), four(p[..., E:E + N]), four(p[..., E + N:]), f(m.skip), f(xz[..., E:]),
                    f(m.bias), True, None, None)
    ref.check("u", u, want[0], want[1], m.ty)
    ref.check("state", s, want[2], want[3], torch.float32)
    want = bref.block(f(o), f(h), True, f(m.w_post), f(m.gate), 1.0, 1.0, True, f(m.w_pre), False, EPS)
    ref.check("h'", h1, want[0], want[1], m.ty)
    ref.check("y'", y1, want[2], want[3], m.ty)


def backward(m, h, forward_out, dy1, dh1):
    """The block's gradients by the operators' own, and those of its projections."""
    E, N = m.E, m.N
    y, (xz, x, p, u), o, _, _, h1, _ = forward_out
    d_o, dh, *_ = la.block_norm_bwd(o, h1, dy1, dh1, **m.seam())
    du = d_o @ m.w_out.t()
    dxz, dp = torch.empty_like(xz), torch.empty_like(p)
    dx, _, dA, _, _, dskip, _, dbias, _ = la.ssm_bwd(
        x, p[..., :E], m.A, p[..., E:E + N], p[..., E + N:], du, skip=m.skip, gate=xz[..., E:], dt_bias=m.bias,
        ddt=dp[..., :E], db=dp[..., E:E + N], dc=dp[..., E + N:], dgate=dxz[..., E:])
    dx = dx + dp @ m.w_bc.t()
    _, dw, db, _ = la.short_conv_bwd(xz[..., :E], m.conv_w, dx, bias=m.conv_b, dx=dxz[..., :E])
    dy = dxz @ m.w_in.t()
    d_first, *_ = la.block_norm_bwd(h, h, dy, None, pre_weight=m.w_pre, eps=EPS, residual_grad=False)
    return dh + d_first, dA, dskip, dbias, dw, db


def test_block_backward_against_differences():
    """The whole block's gradients against differences of it in fp64 (plain forms)."""
    m, (B, T) = Block(D=32, E=48), (2, 40)
    E, N = m.E, m.N
    h = stream(B, T, m.D)
    out = forward(m, h)
    dy1, dh1 = stream(B, T, m.D, seed=5), stream(B, T, m.D, seed=6)
    grads = [ref.f64(t) for t in backward(m, h, out, dy1, dh1)]
    f = ref.f64
    W = {n: f(getattr(m, n)) for n in ("w_in", "w_bc", "w_out", "w_pre", "w_post", "gate")}
    dy1, dh1 = f(dy1), f(dh1)

    def loss(h, A, skip, bias, cw, cb):
        y = bref.block(h, None, False, None, None, 1.0, 1.0, True, W["w_pre"], False, EPS)[2]
        xz = y @ W["w_in"]
        x = bref.conv(xz[..., :E], cw, cb, True, None, None)[0]
        p = x @ W["w_bc"]
        four = lambda t: t.reshape(B, T, 1, N)
        u = bref.ssm(x, p[..., :E], A, four(p[..., E:E + N]), four(p[..., E + N:]), skip, xz[..., E:], bias, True, None,
                     None)[0]
        h1, _, y1, _ = bref.block(u @ W["w_out"], h, True, W["w_post"], W["gate"], 1.0, 1.0, True, W["w_pre"], False, EPS)
        return (y1 * dy1).sum() + (h1 * dh1).sum()

    at = [f(t) for t in (h, m.A, m.skip, m.bias, m.conv_w, m.conv_b)]
    rng = np.random.default_rng(2)
    for i, grad in enumerate(grads):
        v = rng.standard_normal(at[i].shape)
        step = lambda s: loss(*[a + s * v if j == i else a for j, a in enumerate(at)])
        slope = (step(1e-6) - step(-1e-6)) / 2e-6
        # every link in fp32 (its products too): the 2^-12 of the entries is a thousand roundings
        assert abs(slope - (grad * v).sum()) <= 2 ** -12 * np.abs(grad * v).sum() + 1e-4


def test_decoding_continues_the_prefill():
    """Tokens one at a time against the prefill of the whole, its prompts of other lengths
    packed to the right by positions."""
    m, B, T, head = Block(), 3, 60, 40
    h = stream(B, T, m.D)
    _, y = la.block_norm_fwd(h, None, pre_weight=m.w_pre, eps=EPS)
    pad = torch.tensor([0, 7, 33])  # rows in front of the prompt that do not count
    pos = (torch.arange(T) - pad[:, None]).clamp(min=0).to(torch.int32).to(DEV)
    y = torch.where((torch.arange(T) < pad[:, None])[..., None].to(DEV), torch.full_like(y, 5.0), y)
    _, want, cs_T, s_T = m.inner(y, positions=pos)
    _, _, cs, s = m.inner(y[:, :head].contiguous(), positions=pos[:, :head].contiguous())
    for t in range(head, T):
        o = m.step(y[:, t], cs, s)
        torch.cuda.synchronize()
        # both are within the links' bounds of the same values; a thousand roundings of fp32
        assert float((o - want[:, t]).abs().max()) <= 2.0 ** -14 * float(want.abs().max())
    assert float((cs - cs_T).abs().max()) <= 2.0 ** -14 * float(cs_T.abs().max())
    assert float((s - s_T).abs().max()) <= 2.0 ** -14 * float(s_T.abs().max())
    # what the padding holds does not matter
    other = torch.where((torch.arange(T) < pad[:, None])[..., None].to(DEV), torch.full_like(y, -3.0), y)
    _, again, _, s2 = m.inner(other, positions=pos)
    torch.cuda.synchronize()
    for b in range(B):
        assert torch.equal(again[b, int(pad[b]):], want[b, int(pad[b]):])
    assert torch.equal(s2, s_T)


@pytest.mark.parametrize("T", [70, 700])
def test_other_streams_and_graphs(T):
    """The same bits on another stream, and from a captured graph replayed on new inputs."""
    m, B = Block(dtype=torch.bfloat16), 2
    h, dy1, dh1 = (stream(B, T, m.D, torch.bfloat16, seed=k) for k in (1, 5, 6))
    want = forward(m, h)
    grads = backward(m, h, want, dy1, dh1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = forward(m, h)
        got = backward(m, h, out, dy1, dh1)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, grads)) and torch.equal(out[6], want[6])
    static = torch.zeros_like(h)
    with torch.cuda.stream(side):  # warm-up
        backward(m, static, forward(m, static), dy1, dh1)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(m, static)
        got = backward(m, static, out, dy1, dh1)
    static.copy_(h)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, grads)) and torch.equal(out[6], want[6])


def test_a_stream_given_by_hand():
    """stream= of another stream than the current one: the outputs belong to it."""
    m, B, T = Block(), 2, 300
    h = stream(B, T, m.D)
    _, y = la.block_norm_fwd(h, None, pre_weight=m.w_pre, eps=EPS)
    xz = y @ m.w_in
    want, _ = la.short_conv_fwd(xz[..., :m.E], m.conv_w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = la.short_conv_fwd(xz[..., :m.E], m.conv_w, stream=side)
    p = want @ m.w_bc
    torch.cuda.synchronize()
    args = (want, p[..., :m.E], m.A, p[..., m.E:m.E + m.N], p[..., m.E + m.N:])
    a, _ = la.ssm_fwd(*args)
    torch.cuda.synchronize()
    b, _ = la.ssm_fwd(*args, stream=side)
    c, _ = la.block_norm_fwd(h, None, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(a, b) and torch.equal(c, h)
