"""Forms of the attention operators' calls beyond the shapes of test_gpu_attn8.py and test_gpu_xattn.py: plans that no
longer hold."""

import pytest
import torch

from tests.attn_harness import i32

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
