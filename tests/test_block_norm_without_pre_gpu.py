"""block_norm_bwd without a norm before the next block, which reads no h_out (GPU)."""
import pytest
import torch

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("o_type,r_type", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                           (torch.float32, torch.float32)])
@pytest.mark.parametrize("post", [True, False])
def test_no_h_out_is_needed(o_type, r_type, post):
    from retnet_retention_gb300 import _build
    _build.build()
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)
    o, h, dh = r(2, 7, 96).to(o_type), r(2, 7, 96).to(r_type), r(2, 7, 96).to(r_type)
    opts = dict(post_norm=post, post_weight=r(96) if post else None, gate=r(2, 96), scale=0.5, residual_scale=0.75,
                pre_norm=False)
    h_out, _ = la.block_norm_fwd(o, h, **opts)
    want = la.block_norm_bwd(o, h_out, None, dh, **opts)
    got = la.block_norm_bwd(o, None, None, dh, **opts)
    torch.cuda.synchronize()
    assert got[0].dtype == o_type and got[1].dtype == r_type
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(got[1], (0.75 * dh.float()).to(r_type))


def test_h_out_is_needed_with_the_norm():
    o = torch.ones(1, 2, 32, device=DEV)
    with pytest.raises(la.LinAttnError):
        la.block_norm_bwd(o, None, o, None)
