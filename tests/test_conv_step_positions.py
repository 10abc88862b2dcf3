"""short_conv_step with the token's place in its document: the rows of another document, or of
the padding before a short prompt, that the state still holds do not count.  Refusals on the
host (fake pointers, never touched), the rest on the GPU."""
import ctypes

import pytest
import torch

import block_ref as bref
import layer_ref as ref
import retnet_retention_gb300 as la
from test_block_cpu import BAD, CONV_STEP, FAKE, at, lib  # noqa: F401  (lib: the built library)
from test_short_conv_gpu import inputs, plain

DEV = "cuda"


def call(lib, **over):
    a = dict(x=at(0), x1=64, dt=1, w=at(1), b=at(2), B=2, D=64, W=4, flags=1, s=at(3), so=at(5), pos=at(6), y=at(4))
    a.update(over)
    return lib.la_short_conv_step_at(a["x"], a["x1"], a["dt"], a["w"], a["b"], a["B"], a["D"], a["W"], a["flags"],
                                     a["s"], a["pos"], a["so"], a["y"], None)


@pytest.mark.parametrize("over", CONV_STEP + [dict(pos=at(6) + 4), dict(pos=at(4)), dict(pos=at(5) + 16)],
                         ids=lambda d: ",".join(d))
def test_the_step_at_a_position_refuses(lib, over):  # noqa: F811
    assert call(lib, **over) == BAD


def test_no_sequences_touch_nothing(lib):  # noqa: F811
    assert call(lib, B=0, pos=None) == call(lib, B=0) == la.LA_OK


def test_binding_refuses():
    x, w, s = torch.zeros(2, 32), torch.zeros(32, 4), torch.zeros(2, 3, 32)
    with pytest.raises(ValueError, match="CUDA"):
        la.short_conv_step(x, w, s, positions=torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("B,D,W,dt,sliced", [(1, 16, 4, "f32", False), (7, 48, 2, "bf16", True), (256, 4096, 4, "bf16", True),
                                             (1500, 272, 3, "f32", True), (9, 1040, 4, "bf16", False)])
def test_taps_reach_as_far_as_the_position(B, D, W, dt, sliced):
    """A step at a position is a call of one token with it: its bits, and the sum in fp64; NaN and
    infinities in rows out of reach do not pass, the state moves up all the same."""
    x, w, b, s, _, _, _ = inputs((B, 1, D, W, dt, True, True, True, False, sliced))
    pos = torch.arange(B, dtype=torch.int32, device=DEV) % (W + 2) - 1  # -1 .. W
    far = torch.arange(W - 1, 0, -1, device=DEV)[None, :, None] > pos[:, None, None]
    s = torch.where(far, float("nan"), s.float()).to(s.dtype)
    s[:, 0][pos < W - 1] = float("inf")
    want, last = la.short_conv_fwd(x, w, bias=b, state=s, positions=pos[:, None])
    new = torch.empty_like(s)
    y2 = la.short_conv_step(x[:, 0], w, s, bias=b, positions=pos, state_out=new)
    s1 = s.clone()
    y1 = la.short_conv_step(x[:, 0], w, s1, bias=b, positions=pos)
    torch.cuda.synchronize()
    bits = lambda t: t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
    assert torch.equal(y1, y2) and torch.equal(y1, want[:, 0])
    assert torch.equal(bits(s1), bits(new)) and torch.equal(bits(new), bits(last))
    clean = torch.where(far, 0.0, s.float()).to(s.dtype)
    y, bound, _ = bref.conv(plain(x), plain(w), plain(b), True, plain(clean), pos[:, None].cpu().numpy())
    ref.check("y", y1.unsqueeze(1), y, bound, x.dtype)


@pytest.mark.gpu
def test_positions_that_all_reach_change_nothing():
    x, w, b, s, _, _, _ = inputs((5, 1, 80, 4, "bf16", True, True, True, False, False))
    for pos in (3, 1000, 2 ** 31 - 1):
        buf = torch.full((12,), pos, dtype=torch.int32, device=DEV)
        assert torch.equal(la.short_conv_step(x[:, 0], w, s.clone(), bias=b, positions=buf[3:8]),
                           la.short_conv_step(x[:, 0], w, s.clone(), bias=b))
    with pytest.raises(ValueError):
        la.short_conv_step(x[:, 0], w, s, positions=buf[:4])
    with pytest.raises(TypeError):
        la.short_conv_step(x[:, 0], w, s, positions=buf[:5].long())
    with pytest.raises(ValueError):
        la.short_conv_step(x[:, 0], w, s, positions=buf[:10:2])


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_decoding_behind_short_prompts(graph):
    """Prompts of 1, 2, 3 and 9 tokens behind padding that holds NaN, decoded token by token from the
    states the prefill left: convolution and scan, against the same tokens in one call each."""
    head, more, D, N, W = 9, 6, 48, 16, 4
    lens = torch.tensor([1, 2, 3, 9])
    B, T = len(lens), head + more
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)
    x, dt, b, c = r(B, T, D), r(B, T, D) - 2.0, r(B, T, N), r(B, T, N)
    w, A = r(D, W), -torch.rand(D, N, generator=g).to(DEV) - 0.1
    place = torch.arange(T) - (head - lens)[:, None]
    x = torch.where((place < 0)[..., None].to(DEV), float("nan"), x)
    pos = place.clamp(min=0).to(torch.int32).to(DEV)
    # each prompt by itself, no padding
    want = []
    for k in range(B):
        own = slice(head - int(lens[k]), T)
        u, _ = la.short_conv_fwd(x[k:k + 1, own], w)
        want.append(la.ssm_fwd(u, dt[k:k + 1, own], A, b[k:k + 1, own], c[k:k + 1, own])[0][0, int(lens[k]):])
    p = pos[:, :head].contiguous()
    u, cs = la.short_conv_fwd(x[:, :head].contiguous(), w, positions=p)
    _, h = la.ssm_fwd(u, dt[:, :head].contiguous(), A, b[:, :head].contiguous(), c[:, :head].contiguous(), positions=p)
    xt, at_t = x[:, head].clone(), pos[:, head].clone()
    rows = [t[:, head].clone() for t in (dt, b, c)]

    def step():
        v = la.short_conv_step(xt, w, cs, positions=at_t)
        return la.ssm_step(v, rows[0], A, rows[1], rows[2], h)

    if graph:
        keep = cs.clone(), h.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            y = step()
        cs.copy_(keep[0]), h.copy_(keep[1])
    for t in range(more):
        xt.copy_(x[:, head + t]), at_t.copy_(pos[:, head + t])
        for to, of in zip(rows, (dt, b, c)):
            to.copy_(of[:, head + t])
        if graph:
            captured.replay()
        else:
            y = step()
        torch.cuda.synchronize()
        for k in range(B):
            # the same fp32 operations but for the order of a scan's sums: a thousand roundings
            assert bool(torch.isfinite(y[k]).all())
            assert float((y[k] - want[k][t]).abs().max()) <= 2.0 ** -14 * float(want[k].abs().max())
