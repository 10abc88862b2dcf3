"""Calls of the layer operators at the edges of what their documentation allows:
restarts beside channels that have none, and behind decays that are no numbers;
infinities beside entries that do not turn; gradients in slices that interleave;
far positions with large frequencies; positions anywhere in a buffer;
many short sequences, more than 2^32 channels (GPU)."""
from fractions import Fraction

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


def same(a, b):
    """Equal, NaN to NaN."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# ---- scan: a channel beside one that restarts ----------------------------------------

# B, T, D, type: the kernel of short walks, single CTAs, clusters, the backward's wide
# tiles (3 x 2560), long walks of more than a wave
SCANS = [(1, 12, 32, "f32"), (130, 40, 4096, "bf16"), (2, 100, 64, "f32"), (2, 700, 48, "bf16"),
         (1, 5003, 48, "f32"), (1, 5003, 720, "bf16"), (3, 700, 2560, "bf16"), (5, 2500, 8208, "bf16")]


@pytest.mark.parametrize("c", SCANS, ids=lambda c: "x".join(map(str, c)))
def test_a_restart_leaves_the_other_channels_bits(c):
    """The kernel takes another way through a run of rows where one of a warp's channels
    restarts: the others come out of it bit for bit the same, forward and backward."""
    B, T, D, dt = c
    g = torch.Generator().manual_seed(T + D)
    x, dh = (torch.randn(B, T, D, generator=g).to(TYPES[dt]).to(DEV) for _ in range(2))
    h0, dT = (torch.randn(B, D, generator=g).to(DEV) for _ in range(2))
    log_a = -torch.rand(B, T, D, generator=g).to(DEV)
    cut = log_a.clone()
    cut[:, ::7, ::3] = float("-inf")
    (h, hT), (want, last) = la.scan_fwd(x, cut, h0=h0), la.scan_fwd(x, log_a, h0=h0)
    got_b, want_b = (la.scan_bwd(a, want, dh, h0=h0, dh_T=dT) for a in (cut, log_a))
    torch.cuda.synchronize()
    others = torch.arange(D, device=DEV) % 3 != 0
    for a, b in zip((h, hT, *got_b), (want, last, *want_b)):
        assert torch.equal(a[..., others], b[..., others])


# ---- scan: a decay that is no number, then a restart ---------------------------------

@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("gap", [1, 2, 40])
@pytest.mark.parametrize("c", SCANS, ids=lambda c: "x".join(map(str, c)))
def test_a_decay_that_is_no_number_stays_before_the_restart(c, gap, bad):
    """One token's decay is NaN (or infinite), the restart follows in the same run of
    rows or in a later one, and no other channel restarts: from the restart on, nothing
    is left of it; backward nothing before it."""
    B, T, D, dt = c
    at = T // 3
    cut = at + min(gap, T - 2 - at)
    g = torch.Generator().manual_seed(T + D)
    x, dh = (torch.randn(B, T, D, generator=g).to(TYPES[dt]).to(DEV) for _ in range(2))
    h0, dT = (torch.randn(B, D, generator=g).to(DEV) for _ in range(2))
    log_a = -torch.rand(B, T, D, generator=g).to(DEV)
    log_a[:, cut, ::3] = float("-inf")
    clean, last = la.scan_fwd(x, log_a, h0=h0)
    hit = log_a.clone()
    hit[:, at, ::3] = bad
    h, hT = la.scan_fwd(x, hit, h0=h0)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(hT).all()) and torch.equal(hT, last)
    assert torch.equal(h[:, cut:], clean[:, cut:]) and torch.equal(h[:, :at], clean[:, :at])
    others = torch.arange(D, device=DEV) % 3 != 0
    assert torch.equal(h[..., others], clean[..., others])
    assert not bool(torch.isfinite(h[:, at:cut, ::3]).any())
    # backward the walk meets the bad decay first, the restart then at a token before it
    log_a[:, cut, ::3], back = -0.5, at - min(gap, at - 1)
    log_a[:, back, ::3] = float("-inf")
    want = la.scan_bwd(log_a, clean, dh, h0=h0, dh_T=dT)
    hit = log_a.clone()
    hit[:, at, ::3] = bad
    dx, dla, dh0 = la.scan_bwd(hit, clean, dh, h0=h0, dh_T=dT)
    torch.cuda.synchronize()
    assert torch.equal(dh0, want[2])
    assert torch.equal(dx[:, :back], want[0][:, :back]) and torch.equal(dx[:, at:], want[0][:, at:])
    assert torch.equal(dla[:, :back + 1], want[1][:, :back + 1]) and torch.equal(dla[:, at + 1:], want[1][:, at + 1:])
    assert torch.equal(dx[..., others], want[0][..., others]) and torch.equal(dla[..., others], want[1][..., others])
    assert not bool(torch.isfinite(dx[:, back:at, ::3]).any())
    assert not bool(torch.isfinite(dla[:, back + 1:at + 1, ::3]).any())


def test_a_step_drops_what_its_restart_cuts_off():
    x = torch.randn(2, 48, device=DEV)
    h = torch.full((2, 48), float("nan"), device=DEV)
    h[1] = float("inf")
    log_a = torch.full((2, 48), float("-inf"), device=DEV)
    out = la.scan_step(x, log_a, h)
    torch.cuda.synchronize()
    assert torch.equal(out, x) and torch.equal(h, x)


# ---- qk_rotate: entries that do not turn ---------------------------------------------

@pytest.mark.parametrize("interleaved", [True, False], ids=["adjacent", "halves"])
@pytest.mark.parametrize("d,rot", [(64, 32), (80, 16), (48, 0), (256, 240)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_an_entry_that_does_not_turn_stands_alone(d, rot, interleaved, dt):
    """Without the norm an infinity or a NaN among the entries past rot reaches no other
    entry, forward or backward: y = s x there."""
    B, T, H = 2, 5, 3
    g = torch.Generator().manual_seed(d + rot)
    q = torch.randn(B, T, H, d, generator=g).to(TYPES[dt]).to(DEV)
    hurt = q.clone()
    for i, e in enumerate(range(rot, d, 5)):
        hurt[..., e] = (float("inf"), float("nan"), float("-inf"))[i % 3]
    bad = ~torch.isfinite(hurt[0, 0, 0])
    opts = dict(rot=rot, interleaved=interleaved, norm=False, q_scale=-0.5)
    got, want = la.qk_rotate_fwd(hurt, q, **opts)[0], la.qk_rotate_fwd(q, q, **opts)[0]
    torch.cuda.synchronize()
    assert torch.equal(got[..., ~bad], want[..., ~bad])
    assert same(got[..., bad], -0.5 * hurt.transpose(1, 2)[..., bad])
    dy, dk = hurt.transpose(1, 2).contiguous(), q.transpose(1, 2).contiguous()
    got, want = la.qk_rotate_bwd(q, q, dy, dk, **opts)[0], la.qk_rotate_bwd(q, q, dk, dk, **opts)[0]
    torch.cuda.synchronize()
    assert torch.equal(got[..., ~bad], want[..., ~bad])
    assert same(got[..., bad], -0.5 * hurt[..., bad])


# ---- qk_rotate_bwd: gradients in slices that interleave ------------------------------

def interleaved_slices(kind, B, T, H, d):
    """(the whole gradient, its slices for q and k): each head's q, k and v side by side
    in a token's row, the heads first, or the parts of a head kept in separate rows."""
    if kind == "rows":
        row = torch.full((B, T, H, 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
        return row, row[..., 0, :], row[..., 1, :], row[..., 2, :]
    if kind == "heads":
        row = torch.full((B, H, T, 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
        return row, row[..., 2, :].permute(0, 2, 1, 3), row[..., 0, :].permute(0, 2, 1, 3), row[..., 1, :]
    row = torch.full((B, T, 3, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    return row, row[:, :, 1], row[:, :, 2], row[:, :, 0]


@pytest.mark.parametrize("kind", ["rows", "heads", "blocks"])
@pytest.mark.parametrize("B,T,H,d", [(2, 7, 4, 64), (1, 5, 3, 16), (3, 1, 5, 48), (2, 6, 1, 32), (1, 1, 2, 128)])
def test_gradients_into_interleaved_slices(kind, B, T, H, d):
    """What the forward call reads as slices the gradients fill as such: equal to dense
    ones, and the third part of the row keeps what it held."""
    g = torch.Generator().manual_seed(B + T + H + d)
    q, k = (torch.randn(B, T, H, d, generator=g).bfloat16().to(DEV) for _ in range(2))
    gq, gk = (torch.randn(B, H, T, d, generator=g).bfloat16().to(DEV) for _ in range(2))
    w = torch.rand(d, generator=g).to(DEV)
    want = la.qk_rotate_bwd(q, k, gq, gk, q_weight=w, k_weight=w)
    _, dq, dk, rest = interleaved_slices(kind, B, T, H, d)
    got = la.qk_rotate_bwd(q, k, gq, gk, q_weight=w, k_weight=w, dq=dq, dk=dk)
    torch.cuda.synchronize()
    assert got[0] is dq and got[1] is dk
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((rest == 7).all())


# ---- qk_rotate: the angle at far positions with large frequencies --------------------

# pi to 100 digits
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679,
              10 ** 100)


def exact_turn(p, f):
    """cos and sin of p f: the rest of p f over 2 pi in rationals, then in doubles."""
    turns = Fraction(int(p)) * Fraction(float(f)) / (2 * PI)
    rest = float(turns - round(turns)) * 2.0 * np.pi
    return np.cos(rest), np.sin(rest)


@pytest.mark.parametrize("interleaved", [True, False], ids=["adjacent", "halves"])
def test_the_angle_of_far_positions(interleaved):
    """fp32 accuracy at every position and frequency.  The angle loses 2^-32 turns to the
    word that is kept and |p| 2^-63 <= 2^-32 to the table, 2^-28.3 radians; the rest of an
    eighth of a turn is rounded three times (its word, 2 pi and the product: 3 U of at most
    pi / 4), its series add 2 U and leave out 2^-29; so cosine and sine are off by less
    than 5 U, and y by 3 U more for the scale, a product and a sum."""
    freq = [1.0, 7.3, -3.0, 1000.0, 0.5 ** 20, -12345.678, 3.1e6, 10000.0 ** -0.25,
            2.0 ** 40 + 0.123, -1e15 / 7, 2.0 ** 52 + 1, 1e18, 0.0, 5e-324, 1e-12, 2.0 ** 64 * (1 - 2.0 ** -53)]
    pos = [0, 1, -1, 77, 65537, 2 ** 24 + 1, -(2 ** 27) - 5, 2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 12345]
    rot = d = 2 * len(freq)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, len(pos), 2, d, generator=g)
    y = la.qk_rotate_fwd(q.to(DEV), q.to(DEV), positions=torch.tensor([pos], dtype=torch.int32, device=DEV),
                         inv_freq=freq, interleaved=interleaved, norm=False, q_scale=0.75)[0]
    torch.cuda.synchronize()
    c, s = np.array([[exact_turn(p, f) for f in freq] for p in pos]).transpose(2, 0, 1)[:, None, :, None]
    m = np.arange(rot // 2)
    i, j = (2 * m, 2 * m + 1) if interleaved else (m, m + rot // 2)
    x = ref.f64(q)
    want, size = np.empty_like(x), np.empty_like(x)
    want[..., i], want[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    as_out = lambda v: 0.75 * v.transpose(0, 2, 1, 3)
    ref.check("y", y, as_out(want), 8.0 * ref.U * as_out(size), torch.float32)


# ---- qk_rotate: positions anywhere in a buffer ---------------------------------------

@pytest.mark.parametrize("start", [0, 1, 2, 3, 4])
def test_positions_from_the_middle_of_a_buffer(start):
    """A decoder's slice of its position buffer: int32 addresses, any of them, on a side
    stream and in a captured graph that reads what the buffer holds at its replay."""
    g = torch.Generator().manual_seed(6)
    q = torch.randn(6, 1, 3, 64, generator=g).bfloat16().to(DEV)
    buf = torch.randint(0, 5000, (12, 1), generator=g, dtype=torch.int32).to(DEV)
    pos = buf[start:start + 6]
    want = la.qk_rotate_fwd(q, q, positions=pos.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = la.qk_rotate_fwd(q, q, positions=pos, stream=side)
    grads = la.qk_rotate_bwd(q, q, *want, positions=pos)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wantg = la.qk_rotate_bwd(q, q, *want, positions=pos.clone())
    assert all(torch.equal(a, b) for a, b in zip(grads[:2], wantg[:2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = la.qk_rotate_fwd(q, q, positions=pos)
    buf.add_(17)
    graph.replay()
    want = la.qk_rotate_fwd(q, q, positions=pos.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---- scan: many channels -------------------------------------------------------------

def test_more_than_2_24_tiles():
    """2^27 + 3 sequences of 16 channels, a CTA each: every one is walked."""
    B, D = 2 ** 27 + 3, 16
    x = torch.full((B, 1, D), 1.5, dtype=torch.bfloat16, device=DEV)
    h0 = torch.full((B, D), 2.0, device=DEV)
    log_a = torch.full((B, 1, D), -1.0, device=DEV)
    want = torch.tensor(1.5 + 2.0 * np.exp(-1.0)).bfloat16()
    h, hT = la.scan_fwd(x, log_a, h0=h0, out=torch.zeros_like(x), h_out=h0)
    left = int((h != want).sum())
    assert left == 0
    dx, _, dh0 = la.scan_bwd(log_a, h, x, h0=h0, dx=torch.zeros_like(x))
    # dh0 = a x 1.5: expf's 4 U and a rounding
    left = int((dx != 1.5).sum()), int(((dh0 - 1.5 * np.exp(-1.0)).abs() > 8 * ref.U).sum())
    assert left == (0, 0)


@pytest.mark.parametrize("B,D", [(2 ** 28 + 3, 16), (2 ** 27 + 1, 48), (2, 2 ** 31 - 16)])
def test_as_many_channels_as_the_header_allows(B, D):
    """More than 2^32 channels in all, in sequences of an odd number of 16s."""
    x = torch.full((B, 1, D), 1.5, dtype=torch.bfloat16, device=DEV)
    log_a = torch.full((B, 1, D), -1.0, device=DEV)
    h0 = torch.full((B, D), 2.0, device=DEV)
    want = torch.tensor(1.5 + 2.0 * np.exp(-1.0)).bfloat16()
    h, _ = la.scan_fwd(x, log_a, h0=h0, out=torch.zeros_like(x), h_out=h0)
    left = int((h != want).sum())
    assert left == 0
    want = torch.tensor(1.5 + (1.5 + 2.0 * np.exp(-1.0)) * np.exp(-1.0)).bfloat16()
    out = la.scan_step(x[:, 0], log_a[:, 0], h0, out=h[:, 0].zero_())
    left = int((out != want).sum())
    assert left == 0
