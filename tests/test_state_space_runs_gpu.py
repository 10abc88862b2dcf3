"""The loops that only long or large calls reach, entry by entry on varied inputs (GPU): several
runs for a thread of the convolution's gradients, more than four chunks for a warp of the
join."""
import numpy as np
import pytest
import torch

import block_ref as bref
import layer_ref as ref
from test_short_conv_gpu import inputs as conv_inputs
from test_short_conv_gpu import plain as f64
from test_ssm_gpu import inputs as ssm_inputs
from test_state_space_edges_gpu import check_all

la = pytest.importorskip("retnet_retention_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from retnet_retention_gb300 import _build
    _build.build()
    la.library()


@pytest.mark.parametrize("c", [(4, 2003, 4096, 4, "bf16", True, True, True, True, False),
                               (3, 2501, 4096, 3, "f32", False, False, True, True, True)],
                         ids=lambda c: "x".join(map(str, c)))
def test_conv_gradients_of_several_runs_a_thread(c):
    B, T, D, W, _, act = c[:6]
    # places for runs, 4 CTAs of 4 for each SM over the tiles of 128 channels: fewer than the runs of 64 tokens
    places = 4 * ((4 * torch.cuda.get_device_properties(DEV).multi_processor_count + D // 128 - 1) // (D // 128))
    assert places * 64 < B * T
    x, w, b, s, pos, dy, dT = conv_inputs(c)
    dx, dw, db, ds = la.short_conv_bwd(x, w, dy, bias=b, silu=act, state=s, positions=pos, dstate_T=dT)
    torch.cuda.synchronize()
    x, w, b, s, dy, dT, pos = (*(f64(t) for t in (x, w, b, s, dy, dT)), pos.cpu().numpy())
    v = bref.conv_bwd(x, w, b, act, s, pos, dy, dT)
    ref.check("dx", dx, v[0], v[1], dx.dtype)
    ref.check("dstate", ds, v[6], v[7], ds.dtype)
    # The sums over tokens: a thread adds its runs' (at most twice the tokens there are for a place, and a
    # run), the CTA its 4 threads', the last kernel a row of each of its 32 warps and those together.
    chain = (2.0 * B * T / places + 64 + 4 + 32 + 32) * ref.U
    assert chain < 0.5 / (B * T)  # one token's share of the sum, on the mean, shows
    u, size, rows, use = bref._conv(x, w, b, s, pos)
    du, err = dy, np.zeros_like(dy)
    if act:
        _, slope, ops = bref.silu(u)
        du, err = dy * slope, np.abs(dy) * ((W + 2) * ref.U * size + (ops + 2.0) * ref.U)
    size = np.abs(du)
    for j in range(W):
        at = np.where(use[j], rows[:, j:j + T], 0.0)
        share = (size * np.abs(at)).sum((0, 1))
        bound = (err * np.abs(at)).sum((0, 1)) + chain * share
        ref.check(f"dweight {j}", dw[:, j], v[2][:, j], bound, torch.float32)
    if b is not None:
        ref.check("dbias", db, v[4], err.sum((0, 1)) + chain * size.sum((0, 1)), torch.float32)


@pytest.mark.parametrize("c", [(1, 4608, 16, 16, 1, "f32", True, True, True, True, True, False, False),
                               (1, 5301, 16, 8, 1, "bf16", True, True, True, True, True, False, False),
                               (2, 4608, 32, 32, 2, "f32", False, True, False, False, True, False, False)],
                         ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("starts", [(), (1500, 3333)])
def test_scans_of_many_chunks(c, starts):
    B, T, D, N, G = c[:5]
    lib, code = la.library(), la.LA_DTYPE_F32 if c[5] == "f32" else la.LA_DTYPE_BF16
    # more than 64 chunks, so more than 4 for each of the join's 16 warps (the gradients: 64 or 80 tokens each)
    assert T // (64 if T % 64 == 0 else 80) > 64
    state = 4 * B * D * N
    assert lib.la_ssm_workspace_size(B, T, D, N, G, code) > 65 * state
    s, opts, dy, dh_T = ssm_inputs(c)
    if starts:
        opts["positions"] = torch.ones(B, T, dtype=torch.int32, device=DEV)
        for k in starts:
            opts["positions"][B - 1, k] = 0
    y, hT = la.ssm_fwd(**s, **opts)
    grads = la.ssm_bwd(*s.values(), dy, dh_T=dh_T, **opts)
    torch.cuda.synchronize()
    check_all(s, opts, dy, dh_T, y, hT, grads)
