"""The 8-bit paged cache where its runs are many or broken up: copies of scales past 2^31 of them."""

import numpy as np
import pytest
import torch

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
