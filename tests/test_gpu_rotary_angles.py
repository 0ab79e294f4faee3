"""Rotary angles against integers: a position times the frequency as given, modulo a turn, to 2^-27 of a turn."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.attn_harness import FP32, i32

pytestmark = pytest.mark.gpu

# 2 pi to 60 digits
TURN = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def angle(pos, freq):
    """pos freq modulo a turn, in radians within -pi .. pi: exact but for the last conversion."""
    turns = Fraction(int(pos)) * Fraction(float(freq)) / TURN
    return float((turns - round(turns)) * TURN)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_angles_at_any_position_and_frequency(layout):
    """Pairs (1, 0) become (cos, sin): the angle's error, that of sin and cos (one step, 2^-23) and the last rounding."""
    import verify_bs_step_gb300 as vbs
    freq = [1.0, 0.9, 100.0, 1e4, 1e6 + 0.3, -0.5, -777.7, 1e-3, 1e-9, 6.283185307179586, 3.3333, 2.0 ** 40, 0.0, 1e-30, 123456.789, 5.5e-7]
    pos = np.array([0, 1, 2, 3, 1000, 65537, (1 << 24) + 1, 123456789, (1 << 30) + 7, 2 ** 31 - 2, 2 ** 31 - 1])
    rot = 2 * len(freq)
    rope = vbs.Rotary(rot, freqs=freq, layout=layout)
    x = torch.zeros(len(pos), 1, rot, device="cuda")
    if layout == "half":
        x[..., :len(freq)] = 1
    else:
        x[..., ::2] = 1
    got = rope.apply(i32(pos), x)[0].double().cpu().numpy()[:, 0]
    c, s = (got[:, :len(freq)], got[:, len(freq):]) if layout == "half" else (got[:, ::2], got[:, 1::2])
    want = np.array([[angle(p, f) for f in freq] for p in pos])
    bound = 2 * np.pi * 2.0 ** -27 + 3 * FP32
    assert np.abs(c - np.cos(want)).max() < bound and np.abs(s - np.sin(want)).max() < bound, \
        (np.abs(c - np.cos(want)).max(0), np.abs(s - np.sin(want)).max(0))
    rope.close()
