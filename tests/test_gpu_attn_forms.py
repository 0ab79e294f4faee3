"""Forms of the attention operators' calls beyond the shapes of test_gpu_attn8.py and test_gpu_xattn.py: plans that no
longer hold, scores of minus infinity, several tokens of several beams, many sentences, joins of many pieces."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, DT, FP16, FP16_FLOOR, Decode, check_rows, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def test_a_plan_does_not_outlive_its_tables():
    """After every call that may change the tables attend refuses until they have been planned again."""
    import verify_bs_step_gb300 as vbs
    kv = vbs.PagedKV8(1, 2, 1, 1, 16, heads=1, blocks_per_sentence=8, max_blocks=4, block=4)
    bs = vbs.BeamSearch(1, 2, 20, max_len=4)
    q = torch.ones(2, 1, 1, 16, device="cuda", dtype=torch.bfloat16)
    ctx = i32([3, 3])
    kv.build(i32([3]))
    x = torch.ones(3, 1, 16, device="cuda")
    kv.append(0, x, x, kv.build(i32([3]), 3)[0])
    same = i32([0, 1])

    def beam_step():
        bs.step_paged(torch.randn(2, 20, device="cuda").to(torch.bfloat16), kv, 1)
        kv.copy()

    kv.save()
    for change in (lambda: kv.prepare(0), lambda: kv.reorder(same, 1), beam_step, kv.restore,
                   lambda: kv.prefill(3), lambda: kv.build(i32([3]))):
        kv.plan(ctx)
        a = kv.attend(0, q)
        assert torch.equal(a, kv.attend(0, q))       # the step's layers share the plan
        kv.slot_map(i32([0, 0]), i32([1, 1]), 2)     # (what changes no table leaves it)
        kv.table()
        kv.table(), kv.save()
        kv.attend(0, q)
        change()
        with pytest.raises(vbs.VbsError) as e:
            kv.attend(0, q)
        assert e.value.status == vbs.ESTATE
    kv.plan(ctx)
    kv.attend(0, q)
    assert kv.status() == 0
    kv.close()
    bs.close()


@pytest.mark.parametrize("S", [300, 2000])
@pytest.mark.parametrize("n_q,D", [(1, 64), (3, 80), (100, 64), (100, 128), (40, 256)])
def test_scores_of_minus_infinity(n_q, D, S):
    """Positions that score -inf have no weight; where all that a row sees do, softmax is 0 / 0, and only a row that
    sees none gives zeros."""
    import verify_bs_step_gb300 as vbs
    x = vbs.CrossAttention(3, 1, 2, D, max_q=n_q, max_len=S)
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn(3, n_q, 2, D, device="cuda", generator=g).to(torch.bfloat16)
    q[..., 0] = q[..., 0].abs() + 0.5
    kv = torch.randn(3, S, 2, 2, D, device="cuda", generator=g).to(torch.bfloat16)
    k, v = kv[:, :, 0], kv[:, :, 1]
    lens = [S, S - 3, 0]
    k[0, :, 0, 0] = -float("inf")                    # every position of sentence 0's first head
    k[1, ::3, 0, 0] = -float("inf")                  # a third of sentence 1's, the first and whole tiles among them
    k[1, :S // 2, 1, 0] = -float("inf")
    out = x.attend(q, k, v, i32(lens))
    assert out[0, :, 0].isnan().all() and not out[2].any()
    for b, h in ((0, 1), (1, 0), (1, 1)):
        live = (k[b, :lens[b], h, 0] > -float("inf")).cpu()
        kk, vv = (t[b, :lens[b], h].double().cpu()[live] for t in (k, v))
        at = sorted({int(i) for i in np.linspace(0, n_q - 1, 6)})
        check_rows(out[b, at, h].double().cpu(), q[b, at, h].double().cpu(), kk, vv, [len(kk)] * len(at), D ** -0.5, BF16,
                   f"sentence {b} head {h}")
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("spare", [0, 800])
@pytest.mark.parametrize("n_q,W", [(1, 2), (4, 1)])
def test_scores_of_minus_infinity_over_the_cache(n_q, W, spare):
    """The same where a query holds an infinity and every cached key turns it to -inf: segments whole and in pieces."""
    d = Decode("int8", [70, 0, 900 if spare else 300], W, 4, 2, 64, 16, 0, max_q=n_q, spare=spare)
    d.new = lambda n, f=d.new: tuple(t.index_fill_(2, torch.zeros(1, dtype=torch.long, device="cuda"), -1.0) for t in f(n))
    n = int(d.lens.sum())
    d.kv.append(d.layer, *d.new(n), d.kv.build(i32(d.lens), n)[0])
    g = torch.Generator(device="cuda").manual_seed(n_q + spare)
    q = torch.randn(d.R, n_q, 4, 64, device="cuda", generator=g).to(torch.bfloat16)
    good = q.clone()
    q[:, 0, 1, 0] = float("inf")
    d.kv.plan(i32(d.ctx), n_q)
    out = d.kv.attend(d.layer, q)
    for r in range(d.R):
        sees = int(d.ctx[r]) - n_q + 1
        assert (out[r, 0, 1].isnan().all() if sees > 0 else not out[r, 0, 1].any()), (r, sees)
    # the other heads are what they are without it (within the bound: when a warp's rows move their references depends on
    # all of its rows)
    want = d.kv.attend(d.layer, good)
    d.check(want, good)
    out[:, 0, 1] = want[:, 0, 1]
    d.check(out, good)
    d.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("W,n_q,heads,H,D,block,gen", [(2, 2, 2, 2, 64, 16, 7), (4, 8, 4, 2, 128, 16, 11), (3, 5, 6, 2, 80, 8, 9),
                                                       (5, 3, 1, 1, 48, 24, 26), (2, 32, 2, 1, 64, 32, 3), (16, 2, 2, 2, 256, 16, 5)])
@pytest.mark.parametrize("spare", [0, 800])
def test_several_tokens_of_several_beams(fmt, W, n_q, heads, H, D, block, gen, spare):
    """Beams that share pages, each with several new tokens that see their own past: rows with fewer positions than
    tokens, with none, and of other lengths within a sentence."""
    d = Decode(fmt, [40, 0, 3], W, heads, H, D, block, gen, max_q=n_q, seed=W + n_q, spare=spare)
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn(d.R, n_q, heads, D, device="cuda", generator=g).to(torch.bfloat16)
    ragged = np.maximum(d.ctx - np.arange(d.R) % 5 * 3, 0)
    for ctx in (d.ctx, ragged, np.where(np.arange(d.R) % 2, d.ctx, 0)):
        d.kv.plan(i32(ctx), n_q)
        d.check(d.kv.attend(d.layer, q), q, ctx=ctx)
    d.kv.close()


@pytest.mark.parametrize("B", [128, 129, 300])
@pytest.mark.parametrize("S,D,n_q", [(900, 64, 1), (1700, 128, 3)])
def test_many_sentences_of_an_encoder(B, S, D, n_q):
    """More sentences than a CTA of the split kernel has threads, in a tensor too long for whole segments."""
    import verify_bs_step_gb300 as vbs
    H = 2
    x = vbs.CrossAttention(B, 1, H, D, max_q=n_q, max_len=S)
    g = torch.Generator(device="cuda").manual_seed(B)
    q = torch.randn(B, n_q, H, D, device="cuda", generator=g).to(torch.bfloat16)
    kv = torch.randn(B, S, 2, H, D, device="cuda", generator=g).to(torch.bfloat16)
    rng = np.random.default_rng(B)
    for lens in (rng.integers(0, S + 1, size=B), rng.integers(0, 20, size=B), np.where(np.arange(B) == B - 2, S, 0)):
        out = x.attend(q, kv[:, :, 0], kv[:, :, 1], i32(lens))
        assert x.tiles is False
        for b in range(0, B, 1 if B < 200 else 2):
            n = int(lens[b])
            for h in range(H):
                check_rows(out[b, :, h].double().cpu(), q[b, :, h].double().cpu(), kv[b, :n, 0, h].double().cpu(),
                           kv[b, :n, 1, h].double().cpu(), [n] * n_q, D ** -0.5, BF16, f"sentence {b} head {h}")
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,W", [(129, 1), (300, 1), (150, 2)])
def test_many_sentences_of_a_cache(fmt, B, W):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, size=B)
    lens[B // 2] = 700
    d = Decode(fmt, lens, W, 2, 1, 64, 16, 1 if W == 1 else 5, spare=60, seed=B)
    q = torch.randn(d.R, 1, 2, 64, device="cuda").to(torch.bfloat16)
    d.kv.plan(i32(d.ctx), 1)
    d.check(d.kv.attend(d.layer, q), q)
    d.kv.close()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_joins_of_several_hundred_pieces_of_an_encoder(D):
    """One K/V head over 200 thousand positions: more pieces than one warp joins."""
    import verify_bs_step_gb300 as vbs
    S, n_q = 200_003, 5
    x = vbs.CrossAttention(1, 1, 2, D, kv_heads=1, max_q=n_q, max_len=S)
    g = torch.Generator(device="cuda").manual_seed(D)
    q = (torch.randn(1, n_q, 2, D, device="cuda", generator=g) * 2).to(torch.bfloat16)
    kv = torch.randn(1, S, 2, 1, D, device="cuda", generator=g).to(torch.bfloat16)
    kv[0, :, 1] += 1.0                               # sums that do not cancel: the bound is relative to them
    a = x.attend(q, kv[:, :, 0], kv[:, :, 1], i32([S]))
    assert torch.equal(a, x.attend(q, kv[:, :, 0], kv[:, :, 1], i32([S]))) and x.tiles is False
    k, v = kv[0, :, 0, 0].double(), kv[0, :, 1, 0].double()
    p = torch.softmax(torch.einsum("ihd,sd->ihs", q[0].double(), k) * D ** -0.5, -1)
    want, size = p @ v, p @ v.abs()
    # the result's rounding, a weight's two parts, the scores (|s| below 2^6 here: 2^-24 (D + 8) 2^6), and the sums: a
    # chunk of 16 positions a warp at a time, 4 warps, then 300 pieces: fewer than 1000 roundings of partial sums
    bound = BF16 * want.abs() + (BF16 ** 2 + 2.0 ** -17 * (D + 8) / 32 + 1000 * 2.0 ** -24) * size
    assert ((a[0].double() - want).abs() <= bound).all()
    x.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_joins_of_several_hundred_pieces_of_a_cache(fmt):
    import verify_bs_step_gb300 as vbs
    n, D, block = 200_003, 128, 64
    NB = -(-n // block) + 2
    kv = vbs.PagedKV8(1, 1, 1, 1, D, heads=4, blocks_per_sentence=NB, max_blocks=NB, block=block, dtype=DT[fmt])
    slots = kv.build(i32([n]), n)[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(n, 1, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    kv.append(0, k, v + 1.0, slots)
    q = (torch.randn(1, 1, 4, D, device="cuda", generator=g) * 2).to(torch.bfloat16)
    kv.plan(i32([n]), 1)
    a = kv.attend(0, q)
    assert torch.equal(a, kv.attend(0, q)) and kv.status() == 0
    kk, vv = (t[:, 0].double() for t in kv.read(0, slots))
    p = torch.softmax(torch.einsum("hd,sd->hs", q[0, 0].double(), kk) * D ** -0.5, -1)
    want, size = p @ vv, p @ vv.abs()
    # as above with the weights in fp16, and the queries in effect
    bound = BF16 * want.abs() + (2 * FP16 + 2.0 ** -17 * (D + 8) / 32 + 1000 * 2.0 ** -24) * size + n * FP16_FLOOR * vv.abs().max()
    assert ((a[0, 0].double() - want).abs() <= bound).all()
    kv.close()


def test_an_encoder_as_long_as_32_bits_count():
    """2^31 - 1 positions of equal weight: the last ones are seen."""
    import verify_bs_step_gb300 as vbs
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    S, D = (1 << 31) - 1, 8
    kv = torch.zeros(1, S, 1, D, device="cuda", dtype=torch.bfloat16)
    kv[0, -16:] = 2.0 ** 30
    q = torch.zeros(1, 1, 1, D, device="cuda", dtype=torch.bfloat16)
    x = vbs.CrossAttention(1, 1, 1, D, max_len=S)
    for n, want in ((S, 8.0), (S - 4, 6.0), (S - 14, 1.0)):
        out = x.attend(q, kv, kv, i32([n]))
        assert (out == want).all(), (n, out)
    assert x.status() == 0
    x.close()
    del kv
    torch.cuda.empty_cache()
