"""Forms of the attention operators' calls beyond the shapes of test_gpu_attn8.py and test_gpu_xattn.py: plans that no
longer hold, scores of minus infinity."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, Decode, check_rows, i32

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
    q = torch.randn(d.R, n_q, 4, 64, device="cuda").to(torch.bfloat16)
    good = q.clone()
    q[:, 0, 1, 0] = float("inf")
    d.kv.plan(i32(d.ctx), n_q)
    out = d.kv.attend(d.layer, q)
    for r in range(d.R):
        sees = int(d.ctx[r]) - n_q + 1
        assert (out[r, 0, 1].isnan().all() if sees > 0 else not out[r, 0, 1].any()), (r, sees)
    want = d.kv.attend(d.layer, good)
    same = torch.ones(d.R, n_q, 4, dtype=torch.bool, device="cuda")
    same[:, 0, 1] = False
    assert torch.equal(out[same], want[same])
    d.check(want, good)
    d.kv.close()
