"""Prompt attention's items: what rows that are not there hold, blocks that stand for several items, and the check of cu."""

import numpy as np
import pytest
import torch

from tests.attn_harness import i32
from tests.test_gpu_prompt import check, starts, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("two", [False, True])      # row tiles an item
@pytest.mark.parametrize("G,D", [(3, 64), (7, 64), (5, 128), (3, 128), (6, 72), (3, 256)])
def test_rows_that_are_not_there_change_no_bit(G, D, two, causal):
    """Groups that do not fill a row tile, tokens that do not fill an item: equal calls give equal bits, whatever a call
    of large scores before has left in shared memory and TMEM."""
    import verify_bs_step_gb300 as vbs
    per = 128 // G
    N = 2 * per * sms() + 5 * per + 11 if two else 7 * per + 11
    x, y = vbs.PromptAttention(G, D, kv_heads=1), vbs.PromptAttention(1, D)
    cu = i32(starts([N // 2 - 13, 1, N - N // 2], first=6))
    q, k, v = tensors(N, G, 1, D, seed=G)
    want = x.attend(q, k, v, cu, causal=causal)[6:N - 6]
    for seed in range(3):                            # scores of some 10^6, in every row of the tiles of every SM
        big = tensors(300 * sms(), 1, 1, D, seed=seed, mul=3e5)
        for _ in range(2):
            y.attend(*big, i32(starts([300] * sms())), causal=False)
        got = x.attend(q, k, v, cu, causal=causal)[6:N - 6]
        assert torch.equal(got, want), f"{(got != want).sum()} of {got.numel()} differ"
    assert x.tiles and x.status() == 0 and y.status() == 0
    x.close()
    y.close()
