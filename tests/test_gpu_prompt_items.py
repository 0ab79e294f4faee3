"""Prompt attention's items: what rows that are not there hold, blocks that stand for several items, and the check of cu."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, i32
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


def blocks(items):
    """How many items the grid's first blocks stand for, and how many such blocks there are."""
    batch = max(1, items // (16 * sms()))
    return batch, items * 3 // 4 // batch if batch > 1 else 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,H,D,batch,even", [(1, 64, 64, 2, True), (2, 61, 64, 3, False), (1, 129, 8, 4, False), (3, 41, 128, 2, False),
                                              (2, 67, 136, 2, False)])
def test_blocks_that_stand_for_several_items(G, H, D, batch, even, causal):
    """Calls of so many items that the grid's first blocks stand for several each, its last quarter for one; the first
    blocks' items among them that have no request's tokens."""
    import verify_bs_step_gb300 as vbs
    per = 128 // G * (1 if D > 128 else 2)
    tiles = -(-(16 * batch * sms() + 1) // H)
    while (tiles * H * 3 // 4 % batch == 0) != even or blocks(tiles * H)[0] != batch:
        tiles += 1
    N = tiles * per - per // 3
    rng = np.random.default_rng(H)
    lens, first, last = [], 5, N - 3 * per - 7       # behind the last request: three tiles' items and part of one
    while first + sum(lens) < last:
        lens.append(int(min(rng.integers(0, 90), last - first - sum(lens))))
    cu = starts(lens, first)
    q, k, v = tensors(N, G * H, H, D, seed=H)
    x = vbs.PromptAttention(G * H, D, kv_heads=H)
    out = torch.full((N, G * H, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    x.attend(q, k, v, i32(cu), causal=causal, out=out)
    assert x.tiles and x.status() == 0
    assert out[:first].isnan().all() and out[last:].isnan().all() and torch.isfinite(out[first:last]).all()
    heads = [0, 1, G * H // 2, G * H - 1]
    for b in {0, 1, 2, len(lens) - 2, len(lens) - 1, *rng.integers(0, len(lens), 10).tolist()}:
        check(out, q, k, v, cu[b:b + 2], causal, heads=heads, tokens=5, what=str(b))
    # every row of some heads against plain products in fp32.  The result's rounding and that of the weights are of at
    # most max |v| each; 2^-10 of it is for the fp32 sums of up to 90 terms and their scores
    got, bound = out.float().nan_to_num(0.0), (2 * BF16 + 2.0 ** -10) * v.abs().max().item()
    req = torch.searchsorted(torch.tensor(cu[1:], device="cuda"), torch.arange(N, device="cuda"), right=True)
    for h in {*range(0, G * H, 16), G * H - 1}:
        for a in range(first, last, 2048):           # rows a .. e of requests that start up to 90 before
            e, lo, hi = min(a + 2048, last), max(first, a - 90), min(a + 2048 + 90, last)
            s = q[a:e, h].float() @ k[lo:hi, h // G].float().T * D ** -0.5
            sees = req[a:e, None] == req[None, lo:hi]
            if causal:
                sees &= torch.arange(lo, hi, device="cuda")[None] <= torch.arange(a, e, device="cuda")[:, None]
            p = torch.softmax(s.masked_fill(~sees, -float("inf")), 1)
            want = p @ v[lo:hi, h // G].float()
            assert (got[a:e, h] - want).abs().max() < bound, (h, a)
    x.close()


@pytest.mark.parametrize("kv_heads,tokens,batch", [(1, 40, 3), (8, 9000, 7), (64, 20000, 300), (3, 2000, 5000), (1, 300, 300000)])
def test_one_bad_start_among_many_is_told(kv_heads, tokens, batch):
    """Wherever it stands, and whatever CTA works on which tokens."""
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(kv_heads, 64)
    q, k, v = tensors(tokens, kv_heads, kv_heads, 64)
    good = np.sort(np.random.default_rng(batch).integers(0, tokens + 1, batch + 1))
    x.attend(q, k, v, i32(good))
    assert x.status() == 0
    at = {0, 1, batch // 2, batch - 1, batch, min(31, batch), min(32, batch), min(33, batch), min(4864, batch), min(20000, batch)}
    for b in sorted(at):
        for bad in (-1, tokens + 1):
            cu = good.copy()
            cu[b] = bad
            x.attend(q, k, v, i32(cu))
            assert x.status() == vbs.EINVAL, (b, bad)
    x.attend(q, k, v, i32(good))
    assert x.status() == 0
    x.close()
