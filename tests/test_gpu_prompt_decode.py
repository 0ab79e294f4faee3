"""The operators together: the example's decode, every attention checked against the oracle, and against a decode that
keeps nothing."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, check_rows, i32
from tests.test_gpu_attn16 import weight_eps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


@pytest.mark.parametrize("W,D,block", [(4, 64, 16), (3, 32, 8), (1, 128, 24)])
def test_a_decode_attends_to_what_its_prompts_and_cache_hold(W, D, block):
    from examples.prompt_decode import Decode, Decoder
    m = Decoder(vocab=60, layers=2, heads=4, kv_heads=2, D=D, seed=3)
    prompts = [[3], [i % 60 for i in range(150)], [i % 11 for i in range(22)], [i % 7 for i in range(16)]]
    seen = []

    def prompt(x):
        cu = x["cu"].cpu().numpy()
        q, k, v, o = (x[n].double().cpu().numpy() for n in ("q", "k", "v", "out"))
        for b in range(4):
            a, n = cu[b], cu[b + 1] - cu[b]
            at = np.unique(np.linspace(0, n - 1, 9).astype(int))
            for h in range(4):
                check_rows(o[a + at, h], q[a + at, h], k[a:a + n, h // 2], v[a:a + n, h // 2], at + 1, D ** -0.5, BF16,
                           f"prompt {b} head {h}")
        seen.append(x["layer"])

    d = Decode(m, prompts, W=W, steps=14, block=block, observe=prompt)
    assert seen == [0, 1]

    def check(x):
        ctx = x["ctx"].cpu().numpy()
        pool, table = d.kv.pool[:, x["layer"]], d.kv.table().long()
        p = torch.arange(max(1, int(ctx.max())), device="cuda")
        rows = pool[table[:, p // block].clamp(min=0), :, :, (p % block)[None]].double().cpu().numpy()      # [R, T, 2, H, D]
        q, o = x["q"].double().cpu().numpy(), x["out"][:, 0].double().cpu().numpy()
        for r in range(d.R):
            for h in range(4):
                check_rows(o[r, h:h + 1], q[r, h:h + 1], rows[r, :, 0, h // 2], rows[r, :, 1, h // 2], [ctx[r]], D ** -0.5,
                           weight_eps(W * 2, D), f"step {d.t} row {r} head {h}")

    for _ in range(14):
        d.step(check)
        assert d.kv.status() == 0
    seqs, lens, scores = d.bs.finalize()
    assert torch.isfinite(scores).all() and (lens > 0).all()
    assert d.prompt.status() == 0 and d.bs.status() == 0
    # the cache's prompt rows are the prompts' keys and values: a second prompt pass over prompt + what was generated
    # gives the keys that the steps wrote (bf16 rounding of the layers' inputs apart, exactly the same first layer)
    if W == 1:
        b = 1
        tokens = torch.tensor(prompts[b] + seqs[b, 1:int(lens[b])].tolist(), device="cuda")
        n = len(prompts[b])
        _, k, _ = m.qkv(0, m.emb[tokens])
        _, k2 = m.rotary.apply(i32(np.arange(len(tokens))), k, k)
        table = d.kv.table().long()[b]
        p = torch.arange(n, n + min(3, int(lens[b]) - 2), device="cuda")
        held = d.kv.pool[table[p // block], 0, 0, :, p % block]
        # (the product that makes a key may round differently in a batch of another size: one step of bf16 of its terms)
        assert (held.float() - k2[p].float()).abs().max() <= 4 * BF16 * k2[p].float().abs().max()
    d.close()


def test_the_example_runs_and_repeats():
    from examples.prompt_decode import Decode, Decoder
    m = Decoder(vocab=200, heads=4, kv_heads=4, D=32, seed=1)
    runs = []
    for _ in range(2):
        d = Decode(m, [[1, 2, 3], [4]], W=2, steps=9)
        runs.append([x.clone() for x in d.run()])
        assert d.kv.status() == 0 and d.prompt.status() == 0
        d.close()
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert np.isfinite(runs[0][2].cpu().numpy()).all()


def test_a_captured_step():
    """Plan, append and attend in a graph that is replayed with other tokens, positions and lengths."""
    import verify_bs_step_gb300 as vbs
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kv = vbs.PagedKV16(3, 1, 1, 2, 64, heads=4, blocks_per_sentence=8, max_blocks=8, block=16)
        rope = vbs.Rotary(64)
        kv.build(i32([100, 100, 100]))               # room for 100 positions a row
        g = torch.Generator(device="cuda").manual_seed(0)
        kv.pool.copy_(torch.randn(kv.pool.shape, device="cuda", generator=g))
        q, k, v = (torch.randn(3, n, 64, device="cuda", generator=g).to(torch.bfloat16) for n in (4, 2, 2))
        pos, ctx = i32([10, 20, 30]), i32([11, 21, 31])
        slots = torch.tensor([10, 8 * 16 + 20, 16 * 16 + 30], device="cuda")
        q_out, out = torch.zeros_like(q), torch.zeros(3, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
        kv.append(0, k, v, slots, rotary=rope, pos=pos, q=q, q_out=q_out)
        kv.plan(ctx)
        kv.attend(0, q_out.unsqueeze(1), out=out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kv.append(0, k, v, slots, rotary=rope, pos=pos, q=q, q_out=q_out)
            kv.plan(ctx)
            kv.attend(0, q_out.unsqueeze(1), out=out)
        pos.copy_(i32([40, 0, 99]))
        ctx.copy_(i32([41, 1, 100]))
        slots.copy_(torch.tensor([40, 8 * 16, 16 * 16 + 99], device="cuda"))
        q.copy_(q.flip(0))
        k.copy_(k.flip(0))
        graph.replay()
        side.synchronize()
        got, rotated = out.clone(), q_out.clone()
        want_q, _ = kv.append(0, k, v, slots, rotary=rope, pos=pos, q=q)
        kv.plan(ctx)
        want = kv.attend(0, want_q.unsqueeze(1))
        assert torch.equal(rotated, want_q) and torch.equal(got, want) and kv.status() == 0
        kv.close()
        rope.close()
