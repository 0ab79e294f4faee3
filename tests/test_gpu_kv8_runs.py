"""The 8-bit paged cache where its runs are many or broken up: copies of scales past 2^31 of them, pages whose tokens
skipped ones part."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_copy_on_write_of_scales_past_2_31_runs():
    """A half-filled page whose (page, layer, k/v, head) runs lie past 2^31: its copy carries its scales."""
    import verify_bs_step_gb300 as vbs
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    B, W, L, H, D, block, S, MB = 4, 2, 64, 512, 16, 2, 8200, 8172
    kv = vbs.PagedKV8(B, W, L, H, D, heads=H, blocks_per_sentence=S, max_blocks=MB, block=block, dtype=torch.int8)
    assert kv.scales.numel() > 1 << 31
    n = 8170 * block - 1                             # the last page half filled
    kv.build(_i32([0, 0, 0, n]))
    k, v = (torch.randn(1, H, D, device="cuda") * 100 for _ in range(2))
    at = kv.slot_map(_i32([0, 0, 0, n - 1]), _i32([0, 0, 0, 1]), 1)[0]
    for layer in (0, L - 1):
        kv.append(layer, k, v, at)
    want = [kv.read(layer, at) for layer in (0, L - 1)]
    kv.prepare(0)
    rows = kv.slot_map(_i32([0] * 6 + [n - 1] * 2), _i32([0] * 6 + [1] * 2), 2)[0]
    pages = (rows // block).tolist()
    assert pages[0] != pages[1] and min(pages) * L * 2 * H >= 1 << 31
    assert torch.equal(kv.scales[pages[0]], kv.scales[pages[1]])
    for layer, (wk, wv) in zip((0, L - 1), want):
        gk, gv = kv.read(layer, rows)
        for r in range(2):
            assert torch.equal(gk[r], wk[0]) and torch.equal(gv[r], wv[0])
    assert want[0][0].abs().max() > 100 and kv.status() == 0
    kv.close()
    del kv
    torch.cuda.empty_cache()


def _pieces(rng, NB, block, gaps, bad):
    """Slots of some pages, ascending within each: whole runs, every other offset, or with up to `gaps` skipped tokens
    (-1, or `bad`: outside the pool) between neighbours."""
    slots = []
    for page in rng.permutation(NB)[:max(1, NB * 3 // 4)]:
        n = int(rng.integers(1, block + 1))
        offs = np.sort(rng.choice(block, n, replace=False)) if rng.random() < 0.6 else np.arange(block - n, block)
        for o in offs:
            if gaps and rng.random() < 0.2:
                slots += [int(rng.choice([-1, -1, bad]))] * int(rng.integers(1, gaps + 1))
            slots.append(int(page) * block + int(o))
    return np.array(slots, dtype=np.int64)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,block,NB,gaps,dtype,odd", [
    (16, 8, 9, 1, torch.bfloat16, False), (48, 24, 7, 3, torch.float32, False), (128, 16, 12, 2, torch.bfloat16, False),
    (32, 16, 40, 70, torch.bfloat16, False),         # gaps longer than the 32 tokens that a CTA looks at
    (64, 100, 5, 150, torch.float32, True), (80, 5, 30, 40, torch.bfloat16, True), (64, 16, 30, 0, torch.bfloat16, False),
])
def test_skipped_tokens_inside_a_page(fmt, D, block, NB, gaps, dtype, odd):
    """Runs of one page that skipped tokens part are written one after the other, each as the oracle's."""
    import verify_bs_step_gb300 as vbs
    H = 3
    rng = np.random.default_rng(D + block)
    kv = vbs.PagedKV8(1, 1, 1, H, D, heads=H, blocks_per_sentence=NB, max_blocks=NB, block=block, dtype=DT[fmt])
    codes, scales = np.zeros((NB, 2, H, block, D)), np.zeros((NB, 2, H))
    reported = 0
    for turn in range(4):                            # later turns continue the pages of the ones before
        slots = _pieces(rng, NB, block, gaps, NB * block + turn)
        n = len(slots)
        grow = np.exp(rng.standard_normal((n, H, 1)) * 2 + turn)
        flat = torch.empty(1 + 2 * n * H * D, device="cuda", dtype=dtype)
        kv_new = flat[1:] if odd else flat[:-1]      # odd: rows that are loaded element by element
        kv_new.copy_(torch.from_numpy(rng.standard_normal((2, n, H, D)) * grow).flatten())
        k, v = kv_new.view(2, n, H, D)
        kv.append(0, k, v, torch.from_numpy(slots).cuda())
        kept = np.where(slots < NB * block, slots, -1)
        reported = vbs.EINVAL if (slots >= NB * block).any() else 0
        oa.append(codes, scales, k.double().cpu().numpy(), v.double().cpu().numpy(), kept, fmt)
        np.testing.assert_array_equal(kv.scales[:, 0].cpu().numpy(), scales)
        np.testing.assert_array_equal(kv.pool[:, 0].float().cpu().numpy(), codes)
        assert kv.status() == reported
    kv.close()


def test_a_page_in_three_runs():
    """Slots 5, -1, 7 and 9 of one page, growing, shrinking, and with an infinity in the second."""
    import verify_bs_step_gb300 as vbs
    for fmt in ("int8", "e4m3"):
        kv = vbs.PagedKV8(1, 1, 1, 1, 16, heads=1, blocks_per_sentence=2, max_blocks=2, block=16, dtype=DT[fmt])
        codes, scales = np.zeros((2, 2, 1, 16, 16)), np.zeros((2, 2, 1))
        for sizes, status in (((1.0, 40.0, 3e5), 0), ((1e9, 2.0, 3.0), 0), ((1.0, float("inf"), 1e12), vbs.EINPUT)):
            x = torch.randn(4, 1, 16, device="cuda")
            x[0] *= sizes[0]
            x[2, 0, 3:] *= sizes[1]
            x[3] *= sizes[2]
            slots = np.array([21, -1, 23, 25])
            kv.append(0, x, -x, torch.from_numpy(slots).cuda())
            oa.append(codes, scales, x.double().cpu().numpy(), -x.double().cpu().numpy(), slots, fmt)
            np.testing.assert_array_equal(kv.pool[:, 0].float().cpu().numpy(), codes)
            np.testing.assert_array_equal(kv.scales[:, 0].cpu().numpy(), scales)
            assert kv.status() == status
        kv.close()
