"""The attention oracle against closed forms and torch routines, and the library's refusals (CPU)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import attn as oa


def test_tables_of_ragged_requests_by_hand():
    table, nblk, refcnt, stack, top = oa.build_tables([5, 0, 8], W=2, S=3, MB=4, block=4)
    assert table.tolist() == [[0, 1, -1, -1]] * 2 + [[-1] * 4] * 2 + [[6, 7, -1, -1]] * 2
    assert nblk.tolist() == [2, 2, 0, 0, 2, 2] and top.tolist() == [1, 3, 1]
    assert refcnt.tolist() == [2, 2, 0, 0, 0, 0, 2, 2, 0] and stack.tolist() == [2, 1, 0, 5, 4, 3, 8, 7, 6]
    slots, pos, row, cu = oa.slot_map(table, [0, 2, 4], [3, 0, 7], [2, 0, 1], 4, cap=5)
    assert slots.tolist() == [3, 4, 31, -1, -1] and pos.tolist() == [3, 4, 7, -1, -1]
    assert row.tolist() == [0, 0, 4, -1, -1] and cu.tolist() == [0, 2, 2, 3]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scale_is_the_smallest_power_of_two_that_holds_the_page(fmt):
    for amax in (1e-30, 2.0 ** -60, 0.3, 1.0, 127.0, 127.5, 128.0, 448.0, 449.0, 1e6, 1e30):
        e = oa.scale_exponent(amax, fmt)
        assert oa.E_LO <= e <= oa.E_HI
        assert amax <= oa.QMAX[fmt] * 2.0 ** e or e == oa.E_HI
        assert amax > oa.QMAX[fmt] * 2.0 ** (e - 1) or e == oa.E_LO
    assert oa.scale_exponent(0.0, fmt) == oa.E_LO


def test_e4m3_rounding_is_torchs():
    x = np.concatenate([np.linspace(-460, 460, 9001), np.ldexp(np.linspace(-1, 1, 4001), -5)]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oa.quantise(x, "e4m3"), want)


def test_attention_is_torchs_softmax():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, 8, generator=g, dtype=torch.float64) for n in (4, 9, 9))
    seen = [9, 1, 0, 5]
    got = oa.attention(q, k, v, seen, 0.3)
    for i, t in enumerate(seen):
        want = torch.softmax(k[:t] @ q[i] * 0.3, 0) @ v[:t] if t else torch.zeros(8, dtype=torch.float64)
        np.testing.assert_allclose(got[i], want.numpy(), rtol=1e-12, atol=1e-14)


def test_append_in_pieces_ends_like_append_at_once_where_scales_agree():
    rng = np.random.default_rng(0)
    x = np.clip(rng.standard_normal((2, 10, 2, 16)), -3, 3)
    x[:, :, :, 0] = 3.0                             # every token already holds its page's scale
    whole, parts = (np.zeros((2, 2, 2, 8, 16)) for _ in range(2))
    sw, sp = (np.zeros((2, 2, 2)) for _ in range(2))
    slots = np.arange(10)
    oa.append(whole, sw, x[0], x[1], slots, "int8")
    for i in range(10):
        oa.append(parts, sp, x[0, i:i + 1], x[1, i:i + 1], slots[i:i + 1], "int8")
    np.testing.assert_array_equal(sw, sp)
    np.testing.assert_array_equal(whole, parts)


def test_table_calls_refuse_bad_arguments_before_any_launch():
    import verify_bs_step_gb300 as vbs
    from verify_bs_step_gb300 import _build
    _build.build()
    L = vbs.lib()
    p = [ctypes.c_void_p() for _ in range(5)]
    assert L.kv_paged_build(None, None, 0, None, None, None, None) == vbs.EINVAL
    assert L.kv_paged_slots(None, 1, None, None, 0, None, None, None, None) == vbs.EINVAL
    assert L.kv_paged_state(None, *[ctypes.byref(x) for x in p]) == vbs.EINVAL
