"""Attention over the 16-bit cache in pieces: both joins, on either side of the rule between them.

The join gives a row of a segment (a K/V head of a sentence, up to 32 rows) one warp, or, where segments times rows are at
most two a SM, four."""

import pytest
import torch

from tests.attn_harness import i32
from tests.test_gpu_attn16 import Decode16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def check(lens, W, n_q, heads, H, D, seed=0):
    # (pages to spare: whole segments are for caches that bound them to a few units)
    d = Decode16(lens, W, heads, H, D, 16, 0, max_q=n_q, seed=seed, spare=900, L=1, layer=0)
    q = d.q(n_q, heads)
    d.kv.plan(i32(d.ctx), n_q)
    out = d.kv.attend(0, q)
    d.check(out, q)
    assert torch.equal(d.kv.attend(0, q), out)       # equal calls give equal bits
    d.kv.close()


@pytest.mark.parametrize("more", [-1, 0, 1, 9])
@pytest.mark.parametrize("W,n_q,heads,H,D", [(4, 1, 4, 1, 64), (4, 1, 8, 2, 128), (5, 1, 4, 1, 128), (1, 8, 4, 1, 80), (2, 2, 2, 1, 256)])
def test_both_sides_of_the_rule(W, n_q, heads, H, D, more):
    rows = W * n_q * heads // H
    limit = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    B = limit // (rows * H) + more                   # up to `more` = 0 four warps a row
    lens = [33 + (211 * b) % 400 for b in range(B)]
    lens[0], lens[B // 2] = 2100, 0
    check(lens, W, n_q, heads, H, D, seed=B)


@pytest.mark.parametrize("W,n_q,heads,H,D", [(4, 1, 16, 4, 64), (4, 2, 8, 2, 128)])
def test_many_segments(W, n_q, heads, H, D):
    check([40 + 67 * b % 900 for b in range(20)], W, n_q, heads, H, D)


def test_a_segment_of_several_hundred_pieces_among_many():
    """One long row among short ones: four warps share its pieces, also where rows have a warp each."""
    check([40000] + [30 + b for b in range(24)], 4, 1, 4, 1, 64)


@pytest.mark.parametrize("length", [700, 1500, 4000])
@pytest.mark.parametrize("W,n_q,heads,H,D", [(4, 1, 16, 4, 64), (4, 2, 8, 2, 128), (1, 17, 12, 3, 128), (1, 4, 8, 2, 256)])
def test_an_infinity_stays_one_through_the_joins(W, n_q, heads, H, D, length):
    """Of a value that all rows see, in the first, a middle and the last piece of its segment, few pieces and many."""
    G = heads // H
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count // (min(W * n_q * G, 16) * H) + 1   # a warp a row
    d = Decode16([length] + [60] * (B - 1), W, heads, H, D, 16, 0, max_q=n_q, spare=900, L=1, layer=0)
    q = d.q(n_q, heads)
    d.kv.plan(i32(d.ctx), n_q)
    want = d.kv.attend(0, q)
    assert torch.isfinite(want).all()
    pages = d.kv.table()[0].tolist()
    for p in (0, 17, length // 3, length // 2, 2 * length // 3, length - n_q - 40, length - n_q):
        at = (pages[p // 16], 0, 1, H - 1, p % 16, 7)
        old = d.kv.pool[at].clone()
        d.kv.pool[at] = -float("inf")
        out = d.kv.attend(0, q)
        hit = torch.zeros(out.shape, dtype=torch.bool)
        hit[:W, :, (H - 1) * G:, 7] = True
        assert (out[hit] == -float("inf")).all(), (p, out[hit])
        assert torch.equal(out[~hit], want[~hit]), p
        d.kv.pool[at] = old
    assert d.kv.status() == 0
    d.kv.close()
