"""Attention over the 8-bit paged cache against the fp64 oracle on the values the cache holds.

The weights are rounded to fp16 and so, in effect, is each query (a power of two per row takes its
largest element to the top of fp16's range): two fp16 roundings a term.
"""

import numpy as np
import pytest
import torch

from tests.attn_harness import DT, Decode, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def _q(d, n_q, heads, seed=1, mul=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(d.R, n_q, heads, d.D, device="cuda", generator=g) * mul).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,W,heads,H,D,block,gen", [
    ([1], 1, 1, 1, 16, 1, 0),                      # one token
    ([5, 0, 33, 16], 3, 4, 2, 64, 16, 9),          # an empty prompt; half-filled shared pages
    ([70, 41], 4, 8, 2, 128, 16, 20),              # 16 query rows a K/V head
    ([19, 100, 7], 2, 6, 6, 80, 8, 11),            # pages smaller than a tile, an odd head_dim
    ([90], 5, 7, 1, 32, 24, 30),                   # 35 query rows; pages that end inside a tile
    ([40, 65], 2, 4, 2, 256, 32, 5),
    ([12, 200], 16, 2, 1, 48, 64, 3),              # 16 beams
    ([130], 8, 16, 2, 112, 5, 17),                 # 64 query rows; pages of 5
])
def test_beams_match_the_oracle(fmt, lens, W, heads, H, D, block, gen):
    d = Decode(fmt, lens, W, heads, H, D, block, gen, seed=D + W)
    q = _q(d, 1, heads)
    d.kv.plan(i32(d.ctx), 1)
    d.check(d.kv.attend(d.layer, q), q, what=fmt)
    d.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n_q,heads,H,D,block", [(2, 4, 4, 64, 16), (8, 8, 2, 128, 32), (5, 3, 1, 96, 8), (32, 4, 2, 64, 16),
                                                 (16, 8, 1, 128, 64)])
def test_several_new_tokens_see_their_own_past(fmt, n_q, heads, H, D, block):
    lens = [n_q, 3, 150, 0, 64]                    # rows with fewer positions than tokens, and none
    d = Decode(fmt, lens, 1, heads, H, D, block, 0, max_q=n_q, seed=n_q)
    q = _q(d, n_q, heads)
    d.kv.plan(i32(d.ctx), n_q)
    d.check(d.kv.attend(d.layer, q), q)
    d.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_long_rows_are_split_and_joined(fmt):
    for lens, W, heads, H, D, block in (([20011], 1, 4, 1, 128, 64), ([5003, 1, 9000], 2, 2, 1, 64, 16)):
        d = Decode(fmt, lens, W, heads, H, D, block, 2, seed=3)
        for mul in (1.0, 8.0):                     # flat weights, and a few that hold almost everything
            q = _q(d, 1, heads, mul=mul)
            d.kv.plan(i32(d.ctx), 1)
            d.check(d.kv.attend(d.layer, q), q)
        d.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,W,heads,H,D,block,n_q,gen", [
    ([1], 1, 1, 1, 16, 1, 1, 0),
    ([5, 0, 33, 16], 3, 4, 2, 64, 16, 1, 9),
    ([19, 700, 7], 2, 6, 6, 80, 8, 1, 11),
    ([90, 300], 5, 7, 1, 32, 24, 1, 3),
    ([40, 65], 2, 4, 2, 256, 32, 1, 5),
    ([8, 3, 150, 0, 64], 1, 8, 2, 128, 32, 8, 0),
])
def test_short_rows_in_a_cache_with_room_for_long_ones(fmt, lens, W, heads, H, D, block, n_q, gen):
    """What is short but not bound to be: segments in pieces.  The same rows in a cache without that room, where a
    CTA takes a whole one, are held to the same bound."""
    for spare in (0, 800):
        d = Decode(fmt, lens, W, heads, H, D, block, gen, max_q=n_q, seed=D + n_q, spare=spare)
        q = _q(d, n_q, heads)
        d.kv.plan(i32(d.ctx), n_q)
        d.check(d.kv.attend(d.layer, q), q, what=f"{fmt} {spare}")
        d.kv.close()


def test_lengths_of_each_row():
    """ctx_len below what the tables cover, zero in some rows, different within a sentence."""
    d = Decode("e4m3", [37, 50], 4, 4, 2, 64, 16, 10)
    q = _q(d, 1, 4)
    for ctx in ([0, 1, 47, 16, 0, 0, 0, 0], [17, 15, 16, 47, 60, 33, 1, 59], [0] * 8):
        d.kv.plan(i32(ctx), 1)
        d.check(d.kv.attend(d.layer, q), q, ctx=ctx)
    d.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("scale,spread", [(0.0, 0.7), (-0.3, 0.7), (4.0, 0.3), (0.09, 6.0)])
def test_scales_and_pages_of_very_different_size(fmt, scale, spread):
    """Uniform and reversed weights, one-hot weights, and pages whose magnitudes differ by many powers of two."""
    d = Decode(fmt, [75, 30], 2, 4, 2, 64, 8, 9, spread=spread, seed=11)
    q = _q(d, 1, 4) * (1.0 if spread < 2 else 2.0 ** -9)
    d.kv.plan(i32(d.ctx), 1)
    d.check(d.kv.attend(d.layer, q, scale=scale), q, scale=scale)
    d.kv.close()


def test_queries_of_very_different_size():
    d = Decode("int8", [60], 4, 4, 2, 64, 16, 4)
    q = _q(d, 1, 4)
    q[0] *= 2.0 ** 60
    q[1] *= 2.0 ** -60
    q[2] = 0
    q[3, 0, 0, 5:] *= 2.0 ** -12
    d.kv.plan(i32(d.ctx), 1)
    out = d.kv.attend(d.layer, q, scale=0.1)
    q2, o2 = q[1:], out[1:]
    rows = d.rows()
    from tests.attn_harness import FP16, FP16_FLOOR, check_rows
    for r in range(3):
        for h in range(4):
            check_rows(o2[r, :, h].double().cpu(), q2[r, :, h].double().cpu(), rows[r + 1][0][:, h // 2],
                       rows[r + 1][1][:, h // 2], [d.ctx[r + 1]], 0.1, 2 * FP16, f"row {r + 1}", FP16_FLOOR)
    # the huge query picks the key with the largest score alone
    for h in range(4):
        k, v = rows[0][0][:, h // 2], rows[0][1][:, h // 2]
        best = int(np.argmax(k @ q[0, 0, h].double().cpu().numpy()))
        assert torch.equal(out[0, 0, h].double().cpu(), torch.from_numpy(v[best]))
    d.kv.close()


def test_strided_queries_and_outputs():
    d = Decode("int8", [60, 21], 2, 4, 2, 64, 16, 4)
    big = torch.randn(d.R, 1, 3, 4, 64, device="cuda").to(torch.bfloat16)
    q = big[:, :, 1]
    out = torch.full((d.R, 2, 5, 72), 7.0, device="cuda", dtype=torch.bfloat16)
    odd = torch.randn(1 + d.R * 4 * 64, device="cuda").to(torch.bfloat16)[1:].view(d.R, 1, 4, 64)
    for qq in (q, odd):
        view = out[:, 1:, 1:, 1:65]
        d.kv.plan(i32(d.ctx), 1)
        got = d.kv.attend(d.layer, qq, out=view)
        assert got is view
        d.check(view, qq)
        assert (out[:, 0] == 7).all() and (out[:, 1, 0] == 7).all() and (out[:, 1, 1:, 0] == 7).all()
        assert (out[:, 1, 1:, 65:] == 7).all()
    d.kv.close()


def test_two_calls_give_the_same_bits_and_graphs_replay():
    """The same inputs twice, then a captured step replayed on new inputs in place."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _same_bits_and_replay(side)


def _same_bits_and_replay(side):
    d = Decode("e4m3", [700, 90, 0], 4, 8, 2, 128, 16, 12)
    q = _q(d, 1, 8)
    ctx = i32(d.ctx)
    d.kv.plan(ctx, 1)
    a = d.kv.attend(d.layer, q)
    for _ in range(3):
        d.kv.plan(ctx, 1)
        assert torch.equal(a, d.kv.attend(d.layer, q))
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        d.kv.plan(ctx, 1)
        d.kv.attend(d.layer, q, out=out)
    for seed in (5, 6):
        q.copy_(_q(d, 1, 8, seed=seed))
        ctx.copy_(i32(np.maximum(d.ctx - seed, 0)))
        graph.replay()
        torch.cuda.synchronize()
        d.check(out, q, ctx=np.maximum(d.ctx - seed, 0))
    d.kv.close()


def test_cache_offsets_past_32_bits():
    """A pool of more than 2^32 codes: the last pages of the last layer."""
    import verify_bs_step_gb300 as vbs
    L, H, D, block = 32, 8, 128, 16
    NB = (1 << 32) // (L * 2 * H * block * D) + 40
    kv = vbs.PagedKV8(2, 1, L, H, D, heads=H, blocks_per_sentence=NB // 2, max_blocks=NB // 2, block=block,
                      dtype=torch.int8)
    n = NB // 2 * block
    assert kv.pool.numel() > 1 << 32
    kv.build(i32([0, n]))
    rng = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(40, H, D, device="cuda", generator=rng).to(torch.bfloat16) for _ in range(2))
    slots = kv.slot_map(i32([0, n - 40]), i32([0, 40]), 40)[0]
    kv.append(L - 1, k, v, slots)
    kv.scales[:-3, L - 1] = 0                      # the positions before: zero values
    q = torch.randn(2, 1, H, D, device="cuda", generator=rng).to(torch.bfloat16)
    kv.plan(i32([0, n]), 1)
    out = kv.attend(L - 1, q, scale=1.0)
    kk, vv = (t.double() for t in kv.read(L - 1, slots))
    assert not out[0].any() and kv.status() == 0
    s = torch.einsum("hd,thd->ht", q[1, 0].double(), kk)
    p = torch.exp(s)
    want = torch.einsum("ht,thd->hd", p, vv) / (p.sum(1) + (n - 40))[:, None]
    # the weights' rounding, the result's, and the scores': well below 2^-6 of the values' size
    size = torch.einsum("ht,thd->hd", p, vv.abs()) / (p.sum(1) + (n - 40))[:, None]
    assert ((out[1, 0].double() - want).abs() <= 2.0 ** -6 * size).all()
    kv.close()


def test_refusals():
    import verify_bs_step_gb300 as vbs
    kv = vbs.PagedKV8(2, 2, 1, 2, 32, heads=4, max_q=4, blocks_per_sentence=8, max_blocks=4, block=8)
    q = torch.zeros(4, 2, 4, 32, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(vbs.VbsError) as e:
        kv.attend(0, q)                                              # no plan yet
    assert e.value.status == vbs.ESTATE
    for n_q in (0, 5):
        with pytest.raises(vbs.VbsError) as e:
            kv.plan(i32([1] * 4), n_q)
        assert e.value.status == vbs.EINVAL
    for bad in (i32([1] * 3), i32([1] * 4).long(), i32([1] * 8)[::2]):
        with pytest.raises(ValueError):
            kv.plan(bad, 2)
    kv.build(i32([9, 30]))
    kv.plan(i32([0, 9, 30, 32]), 2)                                  # 32 slots are covered
    assert kv.status() == 0
    kv.plan(i32([-1, 17, 33, 32]), 2)
    assert kv.status() == vbs.EINVAL
    for bad in (q[:, :1], q[:3], q.float(), q.transpose(2, 3), q.cpu()):
        with pytest.raises(ValueError):
            kv.attend(0, bad)
    with pytest.raises(ValueError):
        kv.attend(0, q, out=q[..., :16])
    for kw in ({"layer": 1}, {"layer": -1}, {"layer": 0, "scale": float("nan")}, {"layer": 0, "scale": float("inf")}):
        with pytest.raises(vbs.VbsError) as e:
            kv.attend(q=q, **kw)
        assert e.value.status == vbs.EINVAL
    kv.close()


def test_calls_wait_for_pending_copies():
    """Between BeamSearch.step_paged and PagedKV.copy the cache is neither read nor written."""
    import verify_bs_step_gb300 as vbs
    kv = vbs.PagedKV8(1, 2, 1, 1, 16, heads=1, blocks_per_sentence=8, max_blocks=4, block=4)
    bs = vbs.BeamSearch(1, 2, 20, max_len=4)
    kv.build(i32([3]))
    kv.prepare(0)
    k = torch.ones(2, 1, 16, device="cuda")
    slots = kv.slot_map(i32([3, 3]), i32([1, 1]), 2)[0]
    kv.append(0, k, k, slots)
    kv.plan(i32([4, 4]))
    q = torch.ones(2, 1, 1, 16, device="cuda", dtype=torch.bfloat16)
    kv.attend(0, q)
    bs.step_paged(torch.randn(2, 20, device="cuda").to(torch.bfloat16), kv, 1)
    for call in (lambda: kv.append(0, k, k, slots), lambda: kv.read(0, slots), lambda: kv.plan(i32([4, 4])),
                 lambda: kv.attend(0, q)):
        with pytest.raises(vbs.VbsError) as e:
            call()
        assert e.value.status == vbs.ESTATE
    kv.copy()
    kv.plan(i32([4, 4]))
    kv.attend(0, q)
    assert kv.status() == 0
    kv.close()
    bs.close()
