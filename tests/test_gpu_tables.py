"""Block tables and slot maps built from request lengths: parity with the oracle, ragged decodes."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def _cache(B, W, S, MB, block):
    import verify_bs_step_gb300 as vbs
    return vbs.PagedKV(B, W, 1, 1, 8, blocks_per_sentence=S, max_blocks=MB, block=block)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,W,S,MB,block,hi", [
    (1, 1, 1, 1, 1, 1), (3, 4, 9, 7, 4, 28), (8, 5, 20, 14, 16, 200), (1, 2, 300, 300, 64, 19200),
    (1500, 1, 5, 4, 8, 32), (33, 16, 3, 3, 1, 3),
])
def test_build_matches_oracle(B, W, S, MB, block, hi):
    rng = np.random.default_rng(B * 31 + W)
    lens = rng.integers(0, hi + 1, size=B)
    if B > 2:
        lens[0], lens[-1] = 0, hi
    kv = _cache(B, W, S, MB, block)
    total = int(lens.sum())
    cap = total + 7
    out = kv.build(_i32(lens), cap)
    want = oa.build_tables(lens, W, S, MB, block)
    for got, exp in zip(kv.views(), want):
        np.testing.assert_array_equal(got.cpu().numpy(), exp)
    exp = oa.slot_map(want[0], [b * W for b in range(B)], [0] * B, lens, block, cap)
    for got, e in zip(out, exp):
        np.testing.assert_array_equal(got.cpu().numpy(), e)
    assert kv.build(_i32(lens)) is None                       # the tables alone
    np.testing.assert_array_equal(kv.table().cpu().numpy(), want[0])
    # a few positions of every row, of none, and past the middle
    start = rng.integers(0, lens + 1)
    count = np.minimum(rng.integers(0, 9, size=B), lens - start)
    start_r, count_r = np.repeat(start, W), np.repeat(count, W)
    count_r[::2] = 0
    out = kv.slot_map(_i32(start_r), _i32(count_r), int(count_r.sum()))
    exp = oa.slot_map(want[0], list(range(B * W)), start_r, count_r, block, int(count_r.sum()))
    for got, e in zip(out, exp):
        np.testing.assert_array_equal(got.cpu().numpy(), e)
    assert kv.status() == 0
    kv.close()


def test_bad_lengths_and_uncovered_positions_are_reported():
    import verify_bs_step_gb300 as vbs
    kv = _cache(3, 2, 4, 4, 8)
    slots, pos, row, cu = kv.build(_i32([-1, 33, 8]), 40)       # below zero; more than 4 blocks of 8
    assert kv.status() == vbs.EINVAL and kv.status() == 0
    assert cu.tolist() == [0, 0, 0, 8] and slots[:8].tolist() == list(range(64, 72)) and (slots[8:] == -1).all()
    slots, *_ = kv.build(_i32([4, 4, 4]), 6)                     # more tokens than room: the first 6
    assert slots.tolist() == [0, 1, 2, 3, 32, 33] and kv.status() == vbs.EINVAL
    slots, *_ = kv.slot_map(_i32([0, 0, 6]), _i32([1, 0, 4]), 6)  # positions 8 and 9 of a row with one block
    assert slots.tolist() == [0, 70, 71, -1, -1, -1] and kv.status() == vbs.EINVAL
    slots, *_ = kv.slot_map(_i32([-1, 0, 31]), _i32([1, -2, 2]), 5)
    assert (slots == -1).all() and kv.status() == vbs.EINVAL
    with pytest.raises(ValueError):
        kv.build(_i32([1, 2]))
    with pytest.raises(ValueError):
        kv.build(torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        kv.slot_map(_i32([0, 1]), _i32([1, 1]), 4)
    kv.close()


def test_ragged_prompts_decode_like_each_sentence_alone():
    """Prompts of different lengths, several prepared and reordered positions: every row's logical contents
    are those of a cache that holds its sentence alone, prefilled at its own length."""
    import verify_bs_step_gb300 as vbs
    B, W, L, H, D, block, steps = 4, 3, 2, 2, 8, 4, 11
    lens = [5, 0, 8, 3]
    S, MB = 20, 6
    rng = np.random.default_rng(2)
    kv = vbs.PagedKV(B, W, L, H, D, blocks_per_sentence=S, max_blocks=MB, block=block, dtype=torch.float32)
    alone = [vbs.PagedKV(1, W, L, H, D, blocks_per_sentence=S, max_blocks=MB, block=block, dtype=torch.float32)
             for _ in range(B)]
    kv.build(_i32(lens))
    for b in range(B):
        alone[b].prefill(lens[b])

    def write(cache, rows, p, vals):
        tab = cache.table()[rows, p // block].long()
        cache.pool[tab, :, :, :, p % block, :] = vals

    for b in range(B):
        for p in range(lens[b]):
            val = torch.randn(1, L, 2, H, D, device="cuda")
            write(kv, [b * W], p, val)
            write(alone[b], [0], p, val)
    kv.prepare(0)
    for b in range(B):
        alone[b].prepare(lens[b])
    for t in range(steps):
        for b in range(B):
            vals = torch.randn(W, L, 2, H, D, device="cuda")
            write(kv, list(range(b * W, (b + 1) * W)), lens[b] + t, vals)
            write(alone[b], list(range(W)), lens[b] + t, vals)
        par = np.sort(rng.integers(0, W, size=(B, W)))
        kv.reorder(_i32((par + np.arange(B)[:, None] * W).reshape(-1)), t + 1)
        for b in range(B):
            alone[b].reorder(_i32(par[b]), lens[b] + t + 1)
        for b in range(B):
            n = lens[b] + t + 1
            pages = -(-n // block)
            got = kv.pool[kv.table()[b * W:(b + 1) * W, :pages].long()]
            exp = alone[b].pool[alone[b].table()[:, :pages].long()]
            got, exp = (x.permute(0, 2, 3, 4, 1, 5, 6).reshape(W, L, 2, H, pages * block, D)[..., :n, :]
                        for x in (got, exp))
            assert torch.equal(got, exp), (t, b)
    assert kv.status() == 0
    # a position past the table's end is refused on the device, and nothing is lost
    kv.build(_i32([24, 0, 8, 3]))                   # the first sentence fills its table's 6 blocks of 4
    before = kv.table()
    kv.prepare(0)
    assert kv.status() == vbs.EINVAL and torch.equal(before[:W], kv.table()[:W])
    # save and restore keep the lengths
    kv.build(_i32(lens))
    kv.prepare(0)
    kv.save()
    kv.prefill(2)
    kv.restore()
    kv.prepare(1)
    assert kv.status() == 0
    for c in alone + [kv]:
        c.close()


def test_build_on_another_stream_is_ordered_with_it():
    kv = _cache(4, 1, 8, 8, 16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lens = torch.zeros(4, dtype=torch.int32, device="cuda")
        torch.cuda._sleep(2_000_000)
        lens += torch.arange(4, device="cuda", dtype=torch.int32) * 20
        slots, pos, row, cu = kv.build(lens, 120)
        total = cu[-1].clone()
    side.synchronize()
    assert total.item() == 120 and (slots >= 0).all()
    assert kv.status() == 0
    kv.close()


def test_views_outlive_their_cache():
    """The views keep the library's memory: a cache that is closed or collected does not free it under them."""
    import gc
    kv = _cache(2, 1, 3, 3, 8)
    kv.build(_i32([20, 3]))
    views = kv.views()
    kv.close()
    del kv
    gc.collect()
    other = _cache(2, 1, 3, 3, 8)                 # would take the freed memory
    other.build(_i32([0, 24]))
    assert views[0].tolist() == [[0, 1, 2], [3, -1, -1]] and views[4].tolist() == [0, 2]
    del views
    gc.collect()
    assert other.status() == 0
    other.close()
