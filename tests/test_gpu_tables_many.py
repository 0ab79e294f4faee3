"""Block tables and slot maps of more requests than one launch adds up (4096): the sums come from a kernel of their own."""

import numpy as np
import pytest
import torch

from oracle import attn as oa
from tests.attn_harness import i32

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


def _same(got, want):
    for g, e in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), e)


@pytest.mark.parametrize("B,W,S,MB,block,hi", [(4096, 1, 4, 3, 8, 24), (4097, 1, 4, 3, 8, 24), (5000, 2, 7, 3, 16, 40),
                                               (9001, 1, 2, 2, 5, 10), (20000, 1, 1, 1, 4, 3)])
def test_build_and_slot_map(B, W, S, MB, block, hi):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, hi + 1, size=B)
    lens[-1] = hi
    total = int(lens.sum())
    kv = _cache(B, W, S, MB, block)
    want = oa.build_tables(lens, W, S, MB, block)
    first = [b * W for b in range(B)]
    for cap in (total + 13, total, total - 5):       # room to spare, none, and too little
        import verify_bs_step_gb300 as vbs
        out = kv.build(i32(lens), cap)
        _same(kv.views(), want)
        exp = oa.slot_map(want[0], first, [0] * B, lens, block, max(cap, total))
        _same(out[:3], [e[:cap] for e in exp[:3]])
        _same(out[3:], exp[3:])
        assert kv.status() == (vbs.EINVAL if cap < total else 0)
    assert kv.build(i32(lens)) is None
    _same(kv.views(), want)
    for rows in {tuple(first), tuple(range(B * W))}:
        per = len(rows) // B
        start = np.repeat(rng.integers(0, lens + 1), per)
        count = np.minimum(rng.integers(0, 7, size=len(rows)), np.repeat(lens, per) - start)
        n = int(count.sum())
        _same(kv.slot_map(i32(start), i32(count), n + 3), oa.slot_map(want[0], rows, start, count, block, n + 3))
    assert kv.status() == 0
    kv.close()


def test_bad_lengths_among_many():
    import verify_bs_step_gb300 as vbs
    B, block = 4500, 8
    kv = _cache(B, 1, 3, 3, block)
    lens = np.random.default_rng(1).integers(0, 25, size=B)
    bad = lens.copy()
    bad[[0, 1023, 1024, 4499]] = [-1, 25, -(1 << 31), (1 << 31) - 1]
    lens[[0, 1023, 1024, 4499]] = 0
    out = kv.build(i32(bad), int(lens.sum()) + 4)
    assert kv.status() == vbs.EINVAL and kv.status() == 0
    want = oa.build_tables(lens, 1, 3, 3, block)
    _same(kv.views(), want)
    _same(out, oa.slot_map(want[0], range(B), [0] * B, lens, block, int(lens.sum()) + 4))
    start, count = np.zeros(B, dtype=np.int64), lens.copy()
    start[7], count[7] = 20, 5                       # past the table's end
    start[2000], count[2000] = -3, 4
    start[4498], count[4498] = 1 << 30, (1 << 31) - 1
    out = kv.slot_map(i32(start), i32(count), int(lens.sum()))
    assert kv.status() == vbs.EINVAL
    count[[7, 2000, 4498]] = 0
    _same(out, oa.slot_map(want[0], range(B), np.maximum(start, 0), count, block, int(lens.sum())))
    kv.close()


def test_build_of_many_on_another_stream_and_in_a_graph():
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kv = _cache(5000, 1, 2, 2, 16)
        lens = i32(np.full(5000, 3))
        out = kv.build(lens, 20000)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = kv.build(lens, 20000)
        new = np.random.default_rng(5).integers(0, 5, size=5000)
        lens.copy_(i32(new))
        graph.replay()
        torch.cuda.synchronize()
        want = oa.build_tables(new, 1, 2, 2, 16)
        _same(kv.views(), want)
        _same(held, oa.slot_map(want[0], range(5000), [0] * 5000, new, 16, 20000))
        assert out[3][-1].item() == 15000 and kv.status() == 0
        kv.close()
