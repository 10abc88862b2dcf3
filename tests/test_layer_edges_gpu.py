"""Calls of the layer operators at the edges of what their documentation allows:
restarts beside channels that have none (GPU)."""
import pytest
import torch

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


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
