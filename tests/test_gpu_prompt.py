"""Attention of packed prompts to themselves against the fp64 oracle."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, check_rows, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def tensors(N, Hq, H, D, seed=0, mul=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, Hq + 2 * H, D, device="cuda", generator=g)
    x[:, :Hq] *= mul
    x = x.to(torch.bfloat16)
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]


def starts(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)])


def check(out, q, k, v, cu, causal=True, scale=None, tokens=12, heads=None, what=""):
    """A sample of each request's tokens (its ends among them) against the oracle, for some heads.  One weight rounding
    to bf16 a term, in the tiles; the other kernel has none."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    heads = range(Hq) if heads is None else heads
    o, qq, kk, vv = (x.double().cpu().numpy() for x in (out, q, k, v))
    for b in range(len(cu) - 1):
        a, n = int(cu[b]), int(cu[b + 1] - cu[b])
        at = np.unique(np.linspace(0, n - 1, tokens).astype(int)) if n else []
        for h in heads if n else ():
            check_rows(o[a + at, h], qq[a + at, h], kk[a:a + n, h // G], vv[a:a + n, h // G], at + 1 if causal else [n] * len(at),
                       scale, BF16, f"{what} request {b} head {h}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,H,D", [
    ([1], 1, 1, 8), ([5, 0, 130, 1], 2, 2, 64), ([127, 128, 129], 4, 4, 64), ([300], 8, 2, 128), ([33, 600, 64], 8, 1, 128),
    ([70, 200], 6, 2, 80), ([513, 3], 10, 2, 40), ([40] * 9, 7, 1, 64), ([1] * 300, 4, 2, 64), ([257, 255], 1, 1, 128),
    ([0, 0, 31, 0], 16, 1, 128), ([190, 77], 128, 1, 24), ([1025], 3, 3, 96), ([2000, 10], 5, 1, 64),
    ([70, 200], 6, 2, 200), ([33, 12], 40, 2, 256), ([3, 300, 500], 2, 2, 256), ([1, 130], 3, 1, 136)])
def test_matches_the_oracle(lens, Hq, H, D, causal):
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(Hq, D, kv_heads=H)
    cu = starts(lens)
    q, k, v = tensors(int(cu[-1]), Hq, H, D, seed=D + Hq)
    assert x.tiles is None
    out = x.attend(q, k, v, i32(cu), causal=causal)
    assert x.tiles is True
    heads = None if Hq <= 8 else [0, Hq // 2, Hq - 1]
    if len(lens) > 20:
        pick = [0, 1, 63, 64, 65, len(lens) - 1]
        for b in pick:
            check(out, q, k, v, cu[b:b + 2], causal, heads=heads)
    else:
        check(out, q, k, v, cu, causal, heads=heads)
    out = x.attend(q, k, v, i32(cu), causal=causal, scale=-0.7)       # larger scores, a negative scale
    check(out, q, k, v, cu[:4], causal, scale=-0.7, heads=heads)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,H,D,shift", [([5, 0, 90, 1], 2, 2, 64, 1), ([70, 200], 6, 2, 200, 1), ([33, 12], 40, 2, 256, 1),
                                               ([300], 4, 1, 128, 1), ([64], 129, 1, 16, 0), ([3, 50], 3, 1, 136, 1)])
def test_other_layouts(lens, Hq, H, D, shift, causal):
    """More than 128 heads a group, rows 2 bytes off: the other kernel."""
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(Hq, D, kv_heads=H)
    cu = starts(lens)
    N = int(cu[-1])
    q, k, v = tensors(N, Hq, H, D, seed=D)
    if shift:
        flat = torch.empty(N * (Hq + 2 * H) * D + 1, device="cuda", dtype=torch.bfloat16)[1:].view(N, Hq + 2 * H, D)
        flat.copy_(torch.cat([q, k, v], 1))
        q, k, v = flat[:, :Hq], flat[:, Hq:Hq + H], flat[:, Hq + H:]
    out = x.attend(q, k, v, i32(cu), causal=causal)
    assert x.tiles is False
    check(out, q, k, v, cu, causal, heads=None if Hq <= 8 else [0, 17, Hq - 1])
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("Hq,H,D,shift", [(4, 2, 64, 0), (4, 2, 128, 0), (4, 2, 64, 1)])
def test_tokens_of_no_request_are_left(Hq, H, D, shift):
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(Hq, D, kv_heads=H)
    cu = starts([50, 0, 77], first=9)
    N = int(cu[-1]) + 200
    q, k, v = tensors(N, Hq, H, D)
    for t in (q, k, v):
        t[:9] = float("nan")                         # and may hold anything
        t[int(cu[-1]):] = float("inf")
    wide = torch.full((N, Hq + 1, D + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    out = wide[:, :Hq, shift:D + shift]              # strided, and with shift not aligned: stored element by element
    x.attend(q, k, v, i32(cu), out=out)
    check(out, q, k, v, cu)
    assert (wide[:9] == 7).all() and (wide[int(cu[-1]):] == 7).all()
    assert (wide[:, Hq] == 7).all() and (wide[..., D + shift:] == 7).all() and (wide[..., :shift] == 7).all()
    for lens in ([], [0, 0]):                        # nothing to do
        before = wide.clone()
        x.attend(q, k, v, i32(starts(lens)), out=out)
        assert torch.equal(wide, before)
    assert x.attend(q[:0], k[:0], v[:0], i32([0, 0])).shape == (0, Hq, D)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,H", [(64, 4, 1), (128, 2, 2), (192, 2, 1), (8, 3, 3)])
def test_infinities_and_nan_reach_only_those_who_see_them(D, Hq, H, causal):
    """Rows that see no bad position are those of the same call without it; rows that do are not finite where the
    formula is not."""
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(Hq, D, kv_heads=H)
    lens = [100, 333, 40]
    cu = starts(lens)
    q, k, v = tensors(int(cu[-1]), Hq, H, D)
    want = x.attend(q, k, v, i32(cu), causal=causal)
    inf, nan = float("inf"), float("nan")
    bad = {(0, 50, 3): inf, (1, 0, 5): nan, (1, 200, 7): -inf, (1, 332, D - 1): inf, (2, 39, 0): nan}
    v2 = v.clone()
    for (b, p, d), z in bad.items():
        v2[int(cu[b]) + p, 0, d] = z
    out = x.attend(q, k, v2, i32(cu), causal=causal)
    G = Hq // H
    hit = torch.zeros_like(out, dtype=torch.bool)
    for (b, p, d), z in bad.items():
        a = int(cu[b])
        rows = slice(a + p if causal else a, a + lens[b])
        hit[rows, :G, d] = True
        # what a row sees of the bad elements of a dim adds up: infinities of both signs make NaN.  (A weight that has gone
        # to 0 in fp32 makes NaN of an infinity in whole tiles.)
        for t in range(rows.start - a, lens[b]):
            z = sum(x for (b2, p2, d2), x in bad.items() if (b2, d2) == (b, d) and (p2 <= t or not causal))
            got = out[a + t, :G, d]
            assert got.isnan().all() if z != z else ((got == z) | got.isnan()).all(), (b, t, d)
            assert (got == z).all() or z != z or t != p or not causal
    clean = ~hit
    assert torch.isfinite(out[clean]).all()
    check(torch.where(hit, want, out), q, k, v, cu, causal)
    # a key that is not finite makes the scores of those who see it NaN or infinite, and nobody else's
    k2 = k.clone()
    k2[int(cu[1]) + 200, 0, 3] = nan
    out = x.attend(q, k2, v, i32(cu), causal=causal)
    rows = slice(int(cu[1]) + (200 if causal else 0), int(cu[2]))
    assert out[rows, :G].isnan().all()
    out[rows, :G] = want[rows, :G]
    check(out, q, k, v, cu, causal)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("D,Hq,H", [(64, 2, 1), (128, 2, 1), (136, 2, 1)])
def test_scores_of_minus_infinity(D, Hq, H):
    """Positions that score -inf have no weight; a row all of whose positions do is NaN, as the formula."""
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(Hq, D, kv_heads=H)
    cu = starts([20, 400])
    q, k, v = tensors(420, Hq, H, D)
    q[..., 0] = q[..., 0].abs() + 0.5
    k[:7, 0, 0] = -float("inf")                      # the first tokens of request 0, a third of request 1
    k[21:420:3, 0, 0] = -float("inf")
    out = x.attend(q, k, v, i32(cu))
    assert out[:7].isnan().all()
    o, qq, kk, vv = (t.double().cpu().numpy() for t in (out, q, k, v))
    for t in (7, 12, 19, 20, 21, 22, 150, 300, 419):
        a = 0 if t < 20 else 20
        live = np.isfinite(kk[a:t + 1, 0, 0])
        for h in range(Hq):
            check_rows(o[t:t + 1, h], qq[t:t + 1, h], kk[a:t + 1, 0][live], vv[a:t + 1, 0][live], [live.sum()], D ** -0.5, BF16, f"token {t}")
    x.close()


@pytest.mark.parametrize("D,mul", [(64, 40.0), (128, 300.0), (128, 0.0), (256, 100.0)])
def test_extreme_scores(D, mul):
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(2, D)
    cu = starts([290, 3])
    q, k, v = tensors(293, 2, 2, D, mul=mul)
    for scale in (None, 5.0, 0.0):
        out = x.attend(q, k, v, i32(cu), scale=scale)
        check(out, q, k, v, cu, scale=scale, tokens=40)
    # scores that rise all along a request move the reference again and again
    k2 = (k.float().abs() * torch.linspace(0.1, 6, 293, device="cuda")[:, None, None]).to(torch.bfloat16)
    q2 = (q.float().abs() + 0.3).to(torch.bfloat16)
    check(x.attend(q2, k2, v, i32(cu), scale=0.9), q2, k2, v, cu, scale=0.9, tokens=40)
    x.close()


def test_many_requests_and_a_long_one():
    import verify_bs_step_gb300 as vbs
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 5, 9000)                  # more starts than a CTA holds
    lens[4000] = 3001
    cu = starts(lens)
    x = vbs.PromptAttention(2, 64, kv_heads=1)
    q, k, v = tensors(int(cu[-1]), 2, 1, 64)
    out = x.attend(q, k, v, i32(cu))
    for b in [0, 1, 2, 3, 3998, 3999, 4000, 4001, 4096, 4097, 8190, 8191, 8192, 8997, 8998, 8999, *rng.integers(0, 9000, 60)]:
        check(out, q, k, v, cu[b:b + 2], what=str(b))
    assert x.status() == 0
    x.close()


def test_a_long_request():
    import verify_bs_step_gb300 as vbs
    for D, Hq, H in ((128, 8, 1), (64, 3, 1), (256, 1, 1)):
        x = vbs.PromptAttention(Hq, D, kv_heads=H)
        cu = starts([9000, 5000, 1])
        q, k, v = tensors(14001, Hq, H, D, mul=1.5)
        check(x.attend(q, k, v, i32(cu)), q, k, v, cu, tokens=9, heads=[0, Hq - 1])
        x.close()


def test_starts_that_are_not_within_the_tokens():
    """Requests of negative length, before the first or past the last token count as none, and are told."""
    import verify_bs_step_gb300 as vbs
    for D, shift in ((64, 0), (64, 1)):
        x = vbs.PromptAttention(2, D)
        flat = torch.randn(200 * 6 * D + 1, device="cuda").to(torch.bfloat16)[shift:shift + 200 * 6 * D].view(200, 6, D)
        q, k, v = flat[:, :2], flat[:, 2:4], flat[:, 4:]
        for cu in ([0, 50, 300], [-3, 40, 60], [100, 50, 200], [0, 2 ** 31 - 1], [-2 ** 31, 0, 20]):
            out = torch.full((200, 2, D), 7.0, device="cuda", dtype=torch.bfloat16)
            x.attend(q, k, v, i32(cu), out=out)
            assert x.status() == vbs.EINVAL
            for a, e in zip(cu[:-1], cu[1:]):
                if 0 <= a < e <= 200 and sorted(cu) == cu:
                    check(out, q, k, v, [a, e])
            if sorted(cu) == cu:
                good = [(a, e) for a, e in zip(cu[:-1], cu[1:]) if 0 <= a < e <= 200]
                rest = [t for t in range(200) if not any(a <= t < e for a, e in good)]
                assert (out[rest] == 7).all()
        x.close()


def test_streams_graphs_and_repeats():
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(8, 128, kv_heads=2)
    lens = [300, 7, 1000]
    cu = i32(starts(lens))
    q, k, v = tensors(1307, 8, 2, 128)
    want = x.attend(q, k, v, cu)
    assert torch.equal(x.attend(q, k, v, cu), want)  # equal calls give equal bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = x.attend(q, k, v, cu)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    side.synchronize()
    with torch.cuda.stream(side):                    # two contexts at once, on two streams
        y = vbs.PromptAttention(8, 128, kv_heads=2)
    outs = []
    for _ in range(4):
        with torch.cuda.stream(side):
            outs.append(y.attend(q, k, v, cu))
        outs.append(x.attend(q, k, v, cu))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.zeros_like(want)
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            y.attend(q, k, v, cu, out=out)
    cu.copy_(i32(starts([1, 1300, 6])))              # the replay reads the new starts
    q.copy_(q.flip(0))
    g.replay()
    torch.cuda.synchronize()
    check(out, q, k, v, starts([1, 1300, 6]), heads=[0, 7])
    x.close()
    y.close()


def test_strides():
    """Heads before tokens, and K and V of one layout each."""
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(4, 64, kv_heads=2)
    cu = starts([150, 60])
    q, k, v = tensors(210, 4, 2, 64)
    want = x.attend(q, k, v, i32(cu))
    q2 = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    k2 = torch.nn.functional.pad(k, (0, 8))[..., :64]
    out = torch.empty(4, 210, 64, device="cuda", dtype=torch.bfloat16).permute(1, 0, 2)
    assert torch.equal(x.attend(q2, k2, v.contiguous(), i32(cu), out=out), want) and x.tiles
    one = k[:, :1].expand(210, 2, 64)                # one head for all: a stride of 0
    got = x.attend(q, one, v, i32(cu))
    check(got, q, one, v, cu)
    x.close()


def test_refusals():
    import verify_bs_step_gb300 as vbs
    for kw in ({"kv_heads": 3}, {"D": 12}, {"D": 0}, {"D": 264}, {"heads": 0}):
        with pytest.raises(vbs.VbsError):
            vbs.PromptAttention(**{"heads": 4, "D": 64, **kw})
    x = vbs.PromptAttention(4, 64, kv_heads=2)
    q, k, v = tensors(10, 4, 2, 64)
    cu = i32([0, 10])
    bad = [lambda: x.attend(q, k, v, cu.long()), lambda: x.attend(q, k, v, cu.cpu()), lambda: x.attend(q, k, v, cu[:0]),
           lambda: x.attend(q.float(), k, v, cu), lambda: x.attend(q, k[:9], v, cu), lambda: x.attend(q, q, q, cu),
           lambda: x.attend(q, k, v, cu, scale=float("nan")), lambda: x.attend(q, k, v, cu, out=q.float()),
           lambda: x.attend(q[None], k, v, cu), lambda: x.attend(q.cpu(), k, v, cu), lambda: x.attend(q, k, v, cu[None])]
    for f in bad:
        with pytest.raises((ValueError, vbs.VbsError)):
            f()
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("per", [1, 5000, 400000])
def test_any_number_of_empty_requests(per):
    import verify_bs_step_gb300 as vbs
    at = np.array([0, 3, 130, 131, 400, 500])
    cu = np.repeat(at, per)
    x = vbs.PromptAttention(3, 64, kv_heads=1)
    q, k, v = tensors(510, 3, 1, 64)
    out = torch.full((510, 3, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    for causal in (True, False):
        x.attend(q, k, v, i32(cu), causal=causal, out=out)
        check(out, q, k, v, at, causal, what=str(per))
        assert (out[500:] == 7).all()
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("more", [0, 1])
def test_items_of_one_and_of_two_row_tiles(more):
    """One row tile an item, its positions split, up to an SM a pair of them, two beyond: both sides, D of each tile shape."""
    import verify_bs_step_gb300 as vbs
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for D, G in ((64, 2), (128, 1)):
        N = 2 * (128 // G) * sms + more
        cu = starts([N // 3, 1, 0, N // 2, N - N // 3 - 1 - N // 2])
        x = vbs.PromptAttention(G, D, kv_heads=1)
        q, k, v = tensors(N, G, 1, D, seed=more)
        check(x.attend(q, k, v, i32(cu)), q, k, v, cu, tokens=6)
        assert x.tiles and x.status() == 0
        x.close()


def test_two_calls_at_once():
    import verify_bs_step_gb300 as vbs
    lens = np.random.default_rng(3).integers(1, 900, 20)
    cu = starts(lens)
    q, k, v = tensors(int(cu[-1]), 8, 2, 128)
    side = [torch.cuda.Stream() for _ in range(3)]
    xs = []
    for s in side:
        with torch.cuda.stream(s):
            xs.append(vbs.PromptAttention(8, 128, kv_heads=2))
    want = xs[0].attend(q, k, v, i32(cu))
    torch.cuda.synchronize()
    got = []
    cu_ = i32(cu)
    for _ in range(4):
        for s, x in zip(side, xs):
            with torch.cuda.stream(s):
                got.append(x.attend(q, k, v, cu_))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    for x in xs:
        assert x.status() == 0
        x.close()


def test_outputs_whose_rows_are_one_place_are_refused():
    import verify_bs_step_gb300 as vbs
    bf = torch.bfloat16
    x = vbs.PromptAttention(4, 64, kv_heads=2)
    q, k, v = tensors(10, 4, 2, 64)
    wide, tall = torch.zeros(10, 1, 64, device="cuda", dtype=bf).expand(10, 4, 64), torch.zeros(1, 4, 64, device="cuda", dtype=bf).expand(10, 4, 64)
    rope = vbs.Rotary(64)
    kv = vbs.PagedKV16(1, 2, 1, 2, 64, heads=4, blocks_per_sentence=4, max_blocks=4, block=16)
    kv.build(i32([5]))
    kv.plan(i32([5, 5]))
    pos, slots = i32(range(10)), torch.full((10,), -1, device="cuda", dtype=torch.int64)
    q4 = torch.ones(2, 1, 4, 64, device="cuda", dtype=bf)
    for bad in (wide, tall):
        for f in (lambda: x.attend(q, k, v, i32([0, 10]), out=bad), lambda: rope.apply(pos, q, q_out=bad),
                  lambda: rope.apply(pos, q, k, k_out=bad[:, :2]), lambda: kv.append(0, k, v, slots, rotary=rope, pos=pos, q=q, q_out=bad),
                  lambda: kv.append(0, k, v, slots, rotary=rope, pos=pos, k_out=bad[:, :2]), lambda: kv.attend(0, q4, out=bad[:2, None])):
            with pytest.raises(vbs.VbsError):
                f()
    # one row or head has no other to meet
    one = vbs.PromptAttention(1, 64)
    out = torch.zeros(10, 1, 64, device="cuda", dtype=bf)
    one.attend(q[:, :1], k[:, :1], v[:, :1], i32([0, 10]), out=out.as_strided((10, 1, 64), (64, 0, 1)))
    check(out, q[:, :1], k[:, :1], v[:, :1], [0, 10])
    for c in (x, one, kv, rope):
        c.close()


@pytest.mark.parametrize("shift", [0, 1])
def test_offsets_past_32_bits(shift):
    """Rows 2^31 elements and more behind the first, in the tiles and (shifted by one element) in the other kernel; and
    the rotary positions of such rows."""
    import verify_bs_step_gb300 as vbs
    N, wide = 70000, 32768
    buf = torch.zeros(N * wide + 8, device="cuda", dtype=torch.bfloat16)
    rows = buf[shift:shift + N * wide].view(N, wide)
    g = torch.Generator(device="cuda").manual_seed(5)
    rows[:, :256] = torch.randn(N, 256, device="cuda", generator=g).to(torch.bfloat16)
    q, k, v, out = (rows[:, i * 64:i * 64 + 64].unsqueeze(1) for i in (0, 1, 2, 4))
    cu = starts([300] * 10 + [N - 6000] + [300] * 10)
    x = vbs.PromptAttention(1, 64)
    if shift:                                          # (the other kernel: a few tokens behind the 2^31st)
        q, k, v, out, cu = q[68000:], k[68000:], v[68000:], out[68000:], starts([1100, 0, 900])
        assert q.storage_offset() > 2 ** 31
    x.attend(q, k, v, i32(cu), out=out)
    assert x.tiles is (shift == 0)
    check(out, q, k, v, cu, tokens=3)
    if shift == 0:
        rope = vbs.Rotary(64)
        pos = i32(np.arange(N) % 1000)
        want = rope.apply(pos, q.contiguous())[0]
        assert torch.equal(rope.apply(pos, q, q_out=out)[0], want)
        far = rows[:, 1:257].view(N, 4, 64)            # (rows of no 16-byte alignment)
        assert torch.equal(rope.apply(pos, far)[0], rope.apply(pos, far.contiguous())[0])
        rope.close()
    x.close()


def filled(vbs, tokens):
    """PromptAttention with one more request of so many tokens behind the caller's in each call: then items have two row
    tiles."""
    class Filled(vbs.PromptAttention):
        def attend(self, q, k, v, cu, **kw):
            g = torch.Generator(device="cuda").manual_seed(9)
            N = q.shape[0]
            q, k, v = (torch.cat([x, torch.randn(tokens, *x.shape[1:], device="cuda", generator=g).to(x.dtype)]) for x in (q, k, v))
            return super().attend(q, k, v, torch.cat([cu, cu[-1:] + tokens]).contiguous(), **kw)[:N]
    return Filled


@pytest.mark.parametrize("causal", [True, False])   # (of the first two)
@pytest.mark.parametrize("test,args", [
    ("test_matches_the_oracle", ([5, 0, 130, 1], 2, 2, 64)), ("test_matches_the_oracle", ([127, 128, 129], 4, 4, 64)),
    ("test_matches_the_oracle", ([300], 8, 2, 128)), ("test_matches_the_oracle", ([33, 600, 64], 8, 1, 128)),
    ("test_matches_the_oracle", ([70, 200], 6, 2, 80)), ("test_matches_the_oracle", ([1] * 300, 4, 2, 64)),
    ("test_matches_the_oracle", ([2000, 10], 5, 1, 64)), ("test_matches_the_oracle", ([1025], 3, 3, 96)),
    ("test_infinities_and_nan_reach_only_those_who_see_them", (64, 4, 1)),
    ("test_infinities_and_nan_reach_only_those_who_see_them", (128, 2, 2)),
    ("test_infinities_and_nan_reach_only_those_who_see_them", (8, 3, 3)),
    ("test_scores_of_minus_infinity", (64, 2, 1)), ("test_scores_of_minus_infinity", (128, 2, 1)),
    ("test_extreme_scores", (64, 40.0)), ("test_extreme_scores", (128, 300.0)), ("test_extreme_scores", (128, 0.0))])
def test_with_two_row_tiles_an_item(test, args, causal, monkeypatch):
    import verify_bs_step_gb300 as vbs
    Hq, H = args[1:3] if len(args) > 2 else (2, 2)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    monkeypatch.setattr(vbs, "PromptAttention", filled(vbs, 2 * (128 * H // Hq) * (sms // H + 1)))
    globals()[test](*args, causal) if test in ("test_matches_the_oracle", "test_infinities_and_nan_reach_only_those_who_see_them") else \
        globals()[test](*args)


@pytest.mark.parametrize("n", [128, 129, 255, 256, 257, 384, 640, 900])
@pytest.mark.parametrize("D", [64, 128])
def test_positions_split_at_every_count_of_tiles(n, D):
    """Items of 1, 2, 3 .. 8 tiles; rows that see only the first half's, and bad values in either half."""
    import verify_bs_step_gb300 as vbs
    x = vbs.PromptAttention(2, D, kv_heads=1)
    cu = starts([n, 77, n + 40])
    q, k, v = tensors(int(cu[-1]), 2, 1, D, seed=n)
    for causal in (True, False):
        check(x.attend(q, k, v, i32(cu), causal=causal), q, k, v, cu, causal, tokens=30)
    for p in (n // 4, n - 1):
        v2 = v.clone()
        v2[p, 0, 5] = float("inf")
        out = x.attend(q, k, v2, i32(cu))
        assert (out[p, :, 5] == float("inf")).all() and (out[p:n, :, 5] == float("inf")).sum() + out[p:n, :, 5].isnan().sum() == 2 * (n - p)
        out[p:n, :, 5] = x.attend(q, k, v, i32(cu))[p:n, :, 5]
        check(out, q, k, v, cu, tokens=30)
    # a request whose largest scores are in its first half, or all in its second
    for at in (0, n - n // 3):
        k2 = k.clone()
        k2[at:at + n // 3] = (k2[at:at + n // 3].float() * 60).to(torch.bfloat16)
        check(x.attend(q, k2, v, i32(cu)), q, k2, v, cu, tokens=30)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_tokens_of_no_request_in_items_of_two_row_tiles(D, causal):
    """Tokens before the first, behind the last request; items with one row tile of tokens, one of none."""
    import verify_bs_step_gb300 as vbs
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N = 256 * sms + 700
    for first, last in ((100, N - 130), (140, 256 * 20 + 5), (256 * sms, N - 300)):
        cu = starts([(last - first) // 2, last - first - (last - first) // 2], first)
        x = vbs.PromptAttention(1, D)
        q, k, v = tensors(N, 1, 1, D, seed=first)
        v[:first], v[last:], k[:first], k[last:] = float("nan"), float("inf"), float("nan"), float("inf")
        out = torch.full((N, 1, D), 7.0, device="cuda", dtype=torch.bfloat16)
        x.attend(q, k, v, i32(cu), causal=causal, out=out)
        assert (out[:first] == 7).all() and (out[last:] == 7).all() and torch.isfinite(out).all()
        check(out, q, k, v, cu, causal, tokens=8)
        assert x.tiles and x.status() == 0
        x.close()
