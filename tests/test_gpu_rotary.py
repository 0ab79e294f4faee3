"""Rotary positions, alone and on the way into the 16-bit paged cache, against the fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import attn as oa
from tests.attn_harness import BF16, FP32, i32

pytestmark = pytest.mark.gpu

EPS = {torch.float32: FP32, torch.bfloat16: BF16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def check_rotated(got, x, pos, freq, layout, amp=1.0, what="", out_eps=None):
    """got [n, heads, D] against the oracle's rotation of x.

    The angle: the frequency's turns are a double held in units of 2^-64 (with the oracle's own product, some
    2^-51 of p f), what is left of the nearest quarter turn is cut to 2^-34 turns and rounded to fp32 (at most pi / 4
    times 2^-24).  sin and cos are good to one step (2^-23), the amplitude and the two products round once more, and
    the sum once.  The result is rounded to its type."""
    eps = EPS[got.dtype] if out_eps is None else out_eps
    g, xx = got.double().cpu().numpy(), x.double().cpu().numpy()
    pos = np.asarray(pos)
    want = oa.rotate(xx, pos, freq, layout, amp)
    half, rot = len(freq), 2 * len(freq)
    f = np.asarray(freq)
    angle = 0.8 * FP32 + 7 * 2.0 ** -34 + np.abs(pos[:, None, None] * f) * 2.0 ** -51
    a, b = (xx[..., :half], xx[..., half:rot]) if layout == "half" else (xx[..., :rot:2], xx[..., 1:rot:2])
    e = (np.abs(a) + np.abs(b)) * abs(amp) * (angle + 2 * FP32 + 2 * FP32)
    bound = np.zeros_like(want)
    if layout == "half":
        bound[..., :half] = bound[..., half:rot] = e
    else:
        bound[..., :rot:2] = bound[..., 1:rot:2] = e
    bound[..., :rot] += FP32 * np.abs(want[..., :rot])
    bound = bound + eps * (np.abs(want) + bound)
    if out_eps is None:
        bound[..., rot:] = 0                         # not rotated: as they were
    err = np.abs(g - want)
    bad = err > bound
    assert not bad.any(), f"{what}: off by {err[bad].max():.3e}, bound {bound[bad].min():.3e}, at {np.argwhere(bad)[0]}"


def _qkv(n, Hq, H, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, Hq + 2 * H, D, device="cuda", generator=g).to(dtype)
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,Hq,H,D,rot", [(1, 1, 1, 2, 2), (5, 4, 2, 64, 64), (3, 9, 3, 80, 36), (7, 3, 1, 80, 48), (70, 32, 8, 128, 128),
                                          (2, 5, 5, 24, 0), (4, 2, 1, 256, 256), (3, 2, 2, 17, 6), (600, 8, 2, 128, 64),
                                          (9, 70, 1, 16, 16), (5, 3, 2, 48, 32), (4, 6, 1, 7, 6)])
def test_apply_matches_the_oracle(n, Hq, H, D, rot, layout, dtype):
    import verify_bs_step_gb300 as vbs
    rope = vbs.Rotary(D, rot=rot, layout=layout)
    freq = oa.frequencies(rot, 10000.0)
    assert np.allclose(rope.freqs, freq, rtol=1e-15)
    q, k, _ = _qkv(n, Hq, H, D, dtype, seed=D)
    pos = np.random.default_rng(n).integers(0, 5000, n)
    q2, k2 = rope.apply(i32(pos), q, k)
    check_rotated(q2, q, pos, freq, layout, what="q")
    check_rotated(k2, k, pos, freq, layout, what="k")
    q3, none = rope.apply(i32(pos), q)
    assert none is None and torch.equal(q3, q2)
    a, b = q.clone(), k.clone()                      # in place, and into strided memory
    assert rope.apply(i32(pos), a, b, q_out=a, k_out=b)[0] is a
    assert torch.equal(a, q2) and torch.equal(b, k2)
    wide = torch.full((n, Hq + 3, D), 7.0, device="cuda", dtype=dtype)
    rope.apply(i32(pos), q, q_out=wide[:, 1:Hq + 1])
    assert torch.equal(wide[:, 1:Hq + 1], q2) and (wide[:, 0] == 7).all() and (wide[:, Hq + 1:] == 7).all()
    rope.close()


@pytest.mark.parametrize("kw", [{}, {"scaling": "linear", "factor": 4.0}, {"scaling": "base", "factor": 8.0},
                                {"scaling": "parts", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0, "amplitude": 1.25},
                                {"scaling": "parts", "factor": 32.0, "original": 100, "low": 0.5, "high": 9.0}])
def test_scaled_frequencies_at_far_positions(kw):
    import verify_bs_step_gb300 as vbs
    rope = vbs.Rotary(128, base=500000.0, **kw)
    amp = kw.get("amplitude", 1.0)
    freq = oa.frequencies(128, 500000.0, **{x: y for x, y in kw.items() if x != "amplitude"})
    assert np.allclose(rope.freqs, freq, rtol=1e-14)
    pos = np.array([0, 1, 2, 1023, 65537, 1 << 20, (1 << 24) + 1, 123456789, 2 ** 31 - 1])
    q, _, _ = _qkv(len(pos), 3, 1, 128, torch.float32, seed=1)
    got, _ = rope.apply(i32(pos), q)
    check_rotated(got, q, pos, freq, "half", amp)
    if amp == 1.0:
        assert torch.equal(got[0], q[0])             # position 0 turns nothing
    rope.close()


def test_given_frequencies_may_be_any():
    import verify_bs_step_gb300 as vbs
    freq = [0.0, -0.5, 100.0, 2 * np.pi, 1e-30, 3.0, -1e-9, 7.25]
    for layout in ("half", "interleaved"):
        rope = vbs.Rotary(24, rot=16, freqs=freq, layout=layout)
        pos = np.arange(40)
        q, _, _ = _qkv(40, 2, 1, 24, torch.float32)
        got, _ = rope.apply(i32(pos), q)
        check_rotated(got, q, pos, freq, layout)
        rope.close()


def test_skipped_tokens_and_odd_values():
    import verify_bs_step_gb300 as vbs
    rope = vbs.Rotary(64)
    q, k, _ = _qkv(6, 2, 1, 64, torch.bfloat16)
    q[2, 0, 5], q[3, 1, 40] = float("nan"), float("inf")
    out = torch.full((6, 2, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    rope.apply(i32([4, -1, 5, 6, -7, 9]), q, q_out=out)
    assert (out[[1, 4]] == 3).all()
    bad = ~torch.isfinite(out[[0, 2, 3, 5]])
    assert bad.sum() == 4 and bad[1, 0, [5, 37]].all() and bad[2, 1, [8, 40]].all()
    rope.apply(i32([]), q[:0], k[:0])                # no token
    rope.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,Hq,H,D,rot,block,L,layout", [(3, 4, 2, 64, 64, 16, 2, "half"), (2, 6, 3, 80, 30, 8, 1, "interleaved"),
                                                             (5, 8, 1, 128, 128, 24, 3, "interleaved"), (1, 2, 2, 8, 8, 1, 1, "half"),
                                                             (2, 2, 1, 256, 128, 5, 2, "half")])
def test_append_writes_what_it_rotates(batch, Hq, H, D, rot, block, L, layout, dtype):
    import verify_bs_step_gb300 as vbs
    rng = np.random.default_rng(D)
    lens = rng.integers(0, 70, batch)
    lens[-1] = 41
    kv = vbs.PagedKV16(batch, 2, L, H, D, heads=Hq, blocks_per_sentence=80 // block + 3, max_blocks=80 // block + 2, block=block)
    rope = vbs.Rotary(D, rot=rot, layout=layout, base=1000.0)
    kv.pool.fill_(-5.0)
    n = int(lens.sum()) + 3                          # room for more than there is: slot and position -1
    slots, pos, _, _ = kv.build(i32(lens), n)
    q, k, v = _qkv(n, Hq, H, D, dtype, seed=1)
    layer = L - 1
    k_out = torch.full(k.shape, 9.0, device="cuda", dtype=dtype)
    q_out, same = kv.append(layer, k, v, slots, rotary=rope, pos=pos, q=q, q_out=torch.full(q.shape, 9.0, device="cuda", dtype=dtype),
                            k_out=k_out)
    assert same is k_out
    live, freq = slots.cpu().numpy() >= 0, oa.frequencies(rot, 1000.0)
    p = pos.cpu().numpy()[live]
    assert (q_out[~live] == 9).all() and (k_out[~live] == 9).all()
    check_rotated(q_out[live], q[live], p, freq, layout, what="q")
    check_rotated(k_out[live], k[live], p, freq, layout, what="k")
    s = slots[live]
    at = kv.pool[s // block, layer]                  # [n, 2, H, block, D]
    held = at[torch.arange(len(s)), :, :, s % block]
    # from fp32 the cache's value is the same fp32 result, rounded to bf16 once
    assert torch.equal(held[:, 0], k_out[live].to(torch.bfloat16))
    assert torch.equal(held[:, 1], v[live].to(torch.bfloat16))
    mask = torch.ones(kv.pool.shape[:2] + (block,), dtype=torch.bool, device="cuda")
    mask[s // block, layer, s % block] = False
    assert (kv.pool.permute(0, 1, 4, 2, 3, 5)[mask] == -5).all()
    # without rotary: the rows as they are; a slot outside the pool is not written, and told
    kv.append(0, k, v, slots)
    held = kv.pool[s // block, 0][torch.arange(len(s)), :, :, s % block]
    assert torch.equal(held[:, 0], k[live].to(torch.bfloat16)) and torch.equal(held[:, 1], v[live].to(torch.bfloat16))
    assert kv.status() == 0
    before = kv.pool.clone()
    kv.append(0, k[:3], v[:3], torch.tensor([-1, -2, kv.pool.shape[0] * block], device="cuda"))
    assert torch.equal(kv.pool, before) and kv.status() == vbs.EINVAL
    # a token may have a position and no slot: it is rotated, and not written
    q3, _ = kv.append(0, k[:2], v[:2], torch.tensor([-1, -1], device="cuda"), rotary=rope, pos=i32([3, 4]), q=q[:2])
    check_rotated(q3, q[:2], [3, 4], freq, layout, what="no slot")
    assert torch.equal(kv.pool, before)
    kv.close()
    rope.close()


def test_rows_of_any_alignment():
    """The same numbers from rows that start anywhere, 2 bytes on."""
    import verify_bs_step_gb300 as vbs
    rope = vbs.Rotary(64)
    kv = vbs.PagedKV16(1, 1, 1, 2, 64, heads=4, blocks_per_sentence=4, max_blocks=4, block=16)
    q, k, v = _qkv(40, 4, 2, 64, torch.bfloat16)
    flat = torch.empty(40 * 8 * 64 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(40, 8, 64)
    flat.copy_(torch.cat([q, k, v], 1))
    slots, pos = torch.arange(40, device="cuda"), i32(np.arange(40) * 7)
    want, _ = kv.append(0, k, v, slots, rotary=rope, pos=pos, q=q)
    pool = kv.pool.clone()
    kv.pool.zero_()
    got, _ = kv.append(0, flat[:, 4:6], flat[:, 6:], slots, rotary=rope, pos=pos, q=flat[:, :4])
    assert torch.equal(got, want) and torch.equal(kv.pool, pool)
    kv.close()
    rope.close()


def test_another_stream_and_a_graph():
    import verify_bs_step_gb300 as vbs
    rope = vbs.Rotary(128, rot=64)
    q, k, _ = _qkv(300, 8, 2, 128, torch.bfloat16)
    pos = i32(np.arange(300))
    want = rope.apply(pos, q, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = rope.apply(pos, q, k)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.zeros_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(pos, q, q_out=out)
    q.copy_(q.flip(0))
    g.replay()
    assert torch.equal(out, rope.apply(pos, q)[0])
    rope.close()


def test_refusals():
    import verify_bs_step_gb300 as vbs
    for kw in ({"rot": 3}, {"rot": 66}, {"layout": "x"}, {"scaling": "x"}, {"scaling": "linear", "factor": 0.0}, {"base": -1.0},
               {"scaling": "parts", "low": 4.0, "high": 4.0}, {"freqs": [1.0]}, {"freqs": [float("inf")] * 32},
               {"amplitude": float("nan")}, {"rot": 2, "scaling": "base", "factor": 2.0}):
        with pytest.raises((ValueError, vbs.VbsError)):
            vbs.Rotary(64, **kw)
    with pytest.raises(vbs.VbsError):
        vbs.Rotary(257)
    rope = vbs.Rotary(64)
    kv = vbs.PagedKV16(1, 1, 1, 2, 64, heads=4, blocks_per_sentence=4, max_blocks=4, block=16)
    q, k, v = _qkv(4, 4, 2, 64, torch.bfloat16)
    pos, slots = i32(range(4)), torch.arange(4, device="cuda")
    bad = [lambda: rope.apply(pos[:3], q), lambda: rope.apply(pos.long(), q), lambda: rope.apply(pos.cpu(), q),
           lambda: rope.apply(pos, q, k.float()), lambda: rope.apply(pos, q.half()), lambda: rope.apply(pos, q, k_out=k),
           lambda: rope.apply(pos, q, q_out=q.float()), lambda: rope.apply(pos, q.transpose(0, 2)), lambda: rope.apply(pos, q[..., ::2]),
           lambda: kv.append(0, k, v, slots, pos=pos), lambda: kv.append(0, k, v, slots, rotary=rope),
           lambda: kv.append(0, k, v, slots, q=q), lambda: kv.append(0, k, v, slots[:3]), lambda: kv.append(0, k, v, slots.int()),
           lambda: kv.append(0, k, v.float(), slots), lambda: kv.append(1, k, v, slots), lambda: kv.append(-1, k, v, slots),
           lambda: kv.append(0, k, v, slots, rotary=vbs.Rotary(32), pos=pos), lambda: kv.append(0, k[:, :1], v, slots),
           lambda: kv.append(0, k, v, slots, rotary=rope, pos=pos, q_out=q), lambda: kv.append(0, k, v, slots, rotary=rope, pos=pos, q=q[:, :2])]
    for f in bad:
        with pytest.raises((ValueError, vbs.VbsError)):
            f()
    for kw in ({"heads": 3}, {"max_q": 0}, {"max_q": 33}, {"pool": torch.zeros(4, 1, 2, 2, 16, 64, device="cuda")}):
        with pytest.raises((ValueError, vbs.VbsError)):
            vbs.PagedKV16(1, 1, 1, 2, 64, **{"heads": 4, "blocks_per_sentence": 4, "max_blocks": 4, **kw})
    with pytest.raises(vbs.VbsError):
        vbs.PagedKV16(1, 1, 1, 2, 12, heads=4, blocks_per_sentence=4, max_blocks=4)
    kv.close()
    rope.close()
