"""The operators together: the example's decode, its attention checked against the oracle at every step."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, FP16, FP16_FLOOR, check_rows, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


@pytest.mark.parametrize("dtype,W", [(torch.float8_e4m3fn, 4), (torch.int8, 3)])
def test_a_ragged_beam_decode_attends_to_what_its_cache_holds(dtype, W):
    from examples.beam_decode import Decode, Decoder
    g = torch.Generator(device="cuda").manual_seed(5)
    m = Decoder(vocab=60, heads=4, kv_heads=2, D=64, seed=3)
    prompts = [[3], [i % 60 for i in range(21)], [], [i % 7 for i in range(16)]]
    states = torch.randn(4, 23, 256, device="cuda", generator=g).to(torch.bfloat16)
    enc = [23, 1, 9, 0]
    d = Decode(m, prompts, states, i32(enc), W=W, steps=14, eos=2, block=8, dtype=dtype)

    def check(seen):
        t = d.t
        ctx = seen["ctx"].cpu().numpy()
        assert d.kv.status() == 0
        pos = torch.arange(max(1, int(ctx.max())), device="cuda")
        slots = d.kv.table()[:, (pos // 8)].long() * 8 + pos % 8
        k, v = (x.view(d.R, len(pos), 2, 64).double().cpu().numpy()
                for x in d.kv.read(0, slots.clamp(min=0).reshape(-1).contiguous()))
        q, out = seen["q"].double().cpu().numpy(), seen["self"].view(d.R, 4, 64).double().cpu().numpy()
        q2, cross = seen["q2"][:, 0].double().cpu().numpy(), seen["cross"].view(d.R, 4, 64).double().cpu().numpy()
        for r in range(d.R):
            b = r // W
            for h in range(4):
                check_rows(out[r, h:h + 1], q[r, h:h + 1], k[r, :, h // 2], v[r, :, h // 2], [ctx[r]], 0.125,
                           2 * FP16, f"step {t} row {r} head {h}", FP16_FLOOR)
                check_rows(cross[r, h:h + 1], q2[r, h:h + 1], d.enc_k[b, :, h // 2].double().cpu(),
                           d.enc_v[b, :, h // 2].double().cpu(), [enc[b]], 0.125, BF16, f"step {t} row {r} head {h}")

    for _ in range(14):
        d.step(check)
    seqs, lens, scores = d.bs.finalize()
    assert torch.isfinite(scores).all() and (lens > 0).all()
    assert d.kv.status() == 0 and d.cross.status() == 0 and d.bs.status() == 0
    d.close()


def test_the_example_runs_and_repeats():
    from examples.beam_decode import Decode, Decoder
    m = Decoder(vocab=200, heads=4, kv_heads=4, D=32, seed=1)
    states = torch.randn(2, 10, 128, device="cuda").to(torch.bfloat16)
    runs = []
    for _ in range(2):
        d = Decode(m, [[1, 2, 3], [4]], states, i32([10, 3]), W=2, steps=9)
        runs.append([x.clone() for x in d.run()])
        assert d.kv.status() == 0
        d.close()
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert np.isfinite(runs[0][2].cpu().numpy()).all()
