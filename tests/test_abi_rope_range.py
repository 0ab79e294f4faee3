"""Rotary parameters whose numbers leave their type's range are refused (no GPU needed)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def test_frequencies_that_overflow(L):
    import verify_bs_step_gb300 as vbs
    out = (ctypes.c_double * 32)()
    # rot, base, scaling, factor, original, low, high
    for bad in ((64, 1e4, 1, 1e-309, 1, 1, 4),       # freq / factor
                (64, 1e300, 2, 1e300, 1, 1, 4),      # the larger base
                (64, 1e4, 2, 1e-320, 1, 1, 4),       # a base of 0
                (64, 1e4, 3, 1e-309, 1.0, 1, 4)):    # a pair that is stretched
        assert L.rope_frequencies(*bad, out) == vbs.EINVAL, bad
    for good in ((64, 1e300, 0, 1, 1, 1, 4), (64, 1e4, 1, 1e-300, 1, 1, 4), (64, 1e4, 2, 1e100, 1, 1, 4), (64, 1e4, 3, 32.0, 8192, 1, 4)):
        assert L.rope_frequencies(*good, out) == vbs.OK, good
        assert all(0 < x < float("inf") for x in out)


def test_amplitude_past_fp32(L):
    """It is held in fp32, where such a one would be infinite."""
    import verify_bs_step_gb300 as vbs
    ctx, out = ctypes.c_void_p(), (ctypes.c_double * 32)(*([1.0] * 32))
    for amp in (1e39, -3.5e38, float("nan")):
        assert L.rope_init(ctypes.byref(ctx), 64, 64, 0, out, amp) == vbs.EINVAL and not ctx.value
