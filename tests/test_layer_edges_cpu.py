"""Refusals of the layer operators at the edges of what their documentation allows.

Pointers are fake integers that are never touched: each call fails its host checks.
"""
import ctypes

import pytest

import retnet_retention_gb300 as la
from test_layer_cpu import BAD, FAKE, MB, qk_bwd, qk_fwd, s3, scan_call


@pytest.fixture(scope="module")
def lib():
    from retnet_retention_gb300 import _build
    _build.build()
    return la.library()


# a packed gradient row of 4 heads with q, k and v of 64 beside each other: dq first, dk
# behind it
STEP = 3 * 64
ROW = 4 * STEP
INTERLEAVED = dict(Hk=4, dq=FAKE + 6 * MB, dqs=s3(3 * ROW, ROW, STEP), dk=FAKE + 6 * MB + 64 * 2,
                   dks=s3(3 * ROW, ROW, STEP))


@pytest.mark.parametrize("over", [
    dict(dk=FAKE + 6 * MB), dict(dk=FAKE + 6 * MB + 32 * 2), dict(dk=FAKE + 6 * MB + (2 * 64 + 32) * 2),
    dict(dk=FAKE + 6 * MB - 32 * 2), dict(dk=FAKE + 6 * MB + (ROW + 16) * 2),
    dict(dks=s3(3 * ROW, ROW, STEP + 64)), dict(dks=s3(3 * (ROW + 64), ROW + 64, STEP)),
    dict(dks=s3(3 * ROW, ROW, 64)), dict(Hk=2, dks=s3(3 * ROW, ROW, STEP + 8)),
], ids=lambda d: ",".join(d))
def test_interleaved_gradients_that_touch_are_refused(lib, over):
    assert qk_bwd(lib, **dict(INTERLEAVED, **over)) == BAD


@pytest.mark.parametrize("f", [2.0 ** 64, -(2.0 ** 64), 1e300, float("inf"), float("-inf"), float("nan")])
def test_frequencies_without_an_angle_are_refused(lib, f):
    """From 2^64 radians a position on, a double's step is more than the table resolves."""
    freq = (ctypes.c_double * 32)(*([0.5] * 31 + [f]))
    assert qk_fwd(lib, freq=freq) == BAD and qk_bwd(lib, freq=freq) == BAD


def test_the_scans_size_limits(lib):
    """B * D up to 2^33 whatever D is, B * T * D up to 2^44.  A call without tokens and
    with no state to write is accepted and launches nothing."""
    none = dict(T=0, x=None, la=None, h=None, hT=None, dx=None, dla=None, dh0=None)
    for B, D in ((2 ** 29, 16), (2 ** 33 // 48, 48), (2 ** 27, 64), (2 ** 33 // 4112, 4112), (4, 2 ** 31 - 16)):
        for kind in ("fwd", "bwd"):
            assert scan_call(lib, kind, B=B, D=D, **none) == la.LA_OK
            assert scan_call(lib, kind, B=2 ** 33 // D + 1, D=D, **none) == BAD
        assert scan_call(lib, "step", B=2 ** 33 // D + 1, D=D) == BAD
    for kind in ("fwd", "bwd"):
        assert scan_call(lib, kind, B=2 ** 20, T=2 ** 20 + 1, D=16) == BAD
