"""The oracle's rotary positions, pinned by properties and by hand."""

import math

import numpy as np
import pytest

from oracle import attn as oa


def test_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    f = [math.pi / 2, math.pi]
    # position 1: pairs (0, 2) by a quarter turn, (1, 3) by half a turn; the last dim stays
    assert np.allclose(oa.rotate(x, [1], f, "half"), [[[-3.0, -2.0, 1.0, -4.0, 5.0]]])
    assert np.allclose(oa.rotate(x, [1], f, "interleaved"), [[[-2.0, 1.0, -3.0, -4.0, 5.0]]])
    assert np.allclose(oa.rotate(x, [0], f, "half", 2.0), [[[2.0, 4.0, 6.0, 8.0, 5.0]]])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scores_depend_on_the_distance_alone(layout):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 1, 12)), rng.standard_normal((1, 1, 12))
    f = oa.frequencies(12, 10000.0)
    for shift in (0, 5, 1000):
        a, b = oa.rotate(q, [7 + shift], f, layout), oa.rotate(k, [3 + shift], f, layout)
        if shift == 0:
            want = (a * b).sum()
        assert np.isclose((a * b).sum(), want) and np.isclose(np.linalg.norm(a), np.linalg.norm(q))


def test_frequencies():
    assert np.allclose(oa.frequencies(8, 10000.0), [1, 0.1, 0.01, 0.001])
    assert np.allclose(oa.frequencies(8, 10000.0, "linear", 4.0), [0.25, 0.025, 0.0025, 0.00025])
    # the last pair of a larger base is slower by the factor, the first as fast as before
    f = oa.frequencies(8, 10000.0, "base", 4.0)
    assert np.isclose(f[0], 1) and np.isclose(f[-1], 0.001 / 4)
    # by parts: pairs that turn often are left, those that hardly turn are stretched, others lie between
    f = oa.frequencies(64, 10000.0, "parts", 8.0, original=4096, low=1.0, high=4.0)
    g = oa.frequencies(64, 10000.0)
    turns = [4096 * x / (2 * math.pi) for x in g]
    for a, b, t in zip(f, g, turns):
        assert a == b if t >= 4 else np.isclose(a, b / 8) if t <= 1 else b / 8 < a < b


def test_the_library_works_out_the_same_frequencies():
    import ctypes
    import verify_bs_step_gb300 as vbs
    from verify_bs_step_gb300 import _build
    _build.build()
    L = vbs.lib()
    out = (ctypes.c_double * 64)()
    for name, code in vbs.ROPE_SCALINGS.items():
        assert L.rope_frequencies(128, 500000.0, code, 8.0, 8192.0, 1.0, 4.0, out) == vbs.OK
        assert np.allclose(list(out), oa.frequencies(128, 500000.0, name, 8.0, 8192.0, 1.0, 4.0), rtol=1e-14)
