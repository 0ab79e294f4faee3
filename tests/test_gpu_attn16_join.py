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
