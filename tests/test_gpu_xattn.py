"""Cross attention against the fp64 oracle: one weight rounding to bf16 a term (and the result's)."""

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


def _tensors(B, W, n_q, Hq, H, S, D, seed=0, mul=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(B * W, n_q, Hq, D, device="cuda", generator=g) * mul).to(torch.bfloat16)
    kv = torch.randn(B, S, 2, H, D, device="cuda", generator=g).to(torch.bfloat16)
    return q, kv[:, :, 0], kv[:, :, 1]


def _check(out, q, k, v, lens, W, scale=None, sample=None):
    R, n_q, Hq, D = q.shape
    G = Hq // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    for r in range(R):
        b = r // W
        n = max(0, min(int(lens[b]), k.shape[1]))
        for h in range(Hq):
            at = range(n_q) if sample is None else sorted({int(i) for i in np.linspace(0, n_q - 1, sample)})
            at = list(at)
            check_rows(out[r, at, h].double().cpu(), q[r, at, h].double().cpu(), k[b, :n, h // G].double().cpu(),
                       v[b, :n, h // G].double().cpu(), [n] * len(at), scale, BF16, f"row {r} head {h}")


@pytest.mark.parametrize("B,W,n_q,Hq,H,S,D", [
    (1, 1, 1, 1, 1, 1, 8),
    (4, 4, 1, 8, 8, 70, 64),          # a translation step
    (3, 5, 1, 4, 2, 33, 80),
    (2, 16, 1, 2, 1, 300, 128),       # 32 query rows a K/V head
    (2, 2, 7, 6, 2, 19, 40),
    (2, 1, 3, 2, 2, 50, 256),
    (1, 3, 1, 8, 1, 129, 24),
    (2, 1, 33, 3, 1, 65, 64),         # several query tokens
    (3, 1, 130, 2, 2, 200, 64),
    (2, 1, 200, 4, 2, 257, 128),
    (1, 2, 65, 2, 1, 140, 96),
    (1, 1, 129, 2, 2, 128, 192),
    (2, 1, 100, 1, 1, 64, 8),
])
def test_matches_the_oracle(B, W, n_q, Hq, H, S, D):
    import verify_bs_step_gb300 as vbs
    x = vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)
    q, k, v = _tensors(B, W, n_q, Hq, H, S, D, seed=D)
    lens = np.array([S, S // 2, 1, 0][:B])
    out = x.attend(q, k, v, i32(lens))
    _check(out, q, k, v, lens, W, sample=12 if n_q > 12 else None)
    lens = np.array([0, S - 1, S, max(1, S // 3)][:B])               # another call, other lengths, larger scores
    out = x.attend(q, k, v, i32(lens), scale=0.9)
    _check(out, q, k, v, lens, W, scale=0.9, sample=12 if n_q > 12 else None)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("S", [768, 769, 2000])
@pytest.mark.parametrize("W,n_q,Hq,H,D,offset", [
    (4, 1, 8, 8, 64, 0), (2, 1, 3, 1, 80, 0), (1, 5, 2, 2, 128, 0), (5, 8, 2, 2, 64, 1), (3, 12, 1, 1, 256, 0), (2, 20, 2, 1, 128, 1),
    (1, 24, 2, 2, 64, 0),
])
def test_short_sentences_beside_the_longest(S, W, n_q, Hq, H, D, offset):
    """Lengths far below S, on both sides of the size up to which a segment is not split."""
    import verify_bs_step_gb300 as vbs
    lens = [S, 1, 0, 17, S - 1, 16]
    B = len(lens)
    x = vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)
    q, k, v = _tensors(B, W, n_q, Hq, H, S, D, seed=S + D)
    if offset:                                      # not 16-byte aligned: loaded element by element
        k = torch.empty(1 + k.numel(), device="cuda", dtype=torch.bfloat16)[1:].view(k.shape).copy_(k)
    out = x.attend(q, k, v, i32(lens))
    _check(out, q, k, v, lens, W, sample=6)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("n_q", [1, 6, 64, 150])
def test_what_lies_past_a_sentences_end_is_not_used(n_q):
    import verify_bs_step_gb300 as vbs
    B, W, Hq, H, S, D = 3, 2, 4, 2, 150, 64
    x = vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)
    q, k, v = _tensors(B, W, n_q, Hq, H, S, D)
    lens = [131, 0, 16]
    clean = x.attend(q, k, v, i32(lens))
    for b, n in enumerate(lens):
        for t, bad in ((k, float("nan")), (v, float("inf"))):
            t[b, n:] = bad
        v[b, n::2] = float("nan")
        k[b, n::2] = -torch.finfo(torch.bfloat16).max
    out = x.attend(q, k, v, i32(lens))
    assert torch.equal(out, clean) and not out[2:4].any()
    _check(out, q, k, v, lens, W, sample=8)
    x.close()


@pytest.mark.parametrize("n_q", [1, 80])
def test_strides_and_layouts(n_q):
    """Head-major K and V, K and V of different layouts, odd offsets, strided queries and outputs."""
    import verify_bs_step_gb300 as vbs
    B, W, Hq, H, S, D = 2, 3, 4, 2, 90, 64
    x = vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)
    q, k, v = _tensors(B, W, n_q, Hq, H, S, D)
    lens = [90, 37]
    want = x.attend(q, k, v, i32(lens))
    hm = k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    odd = torch.empty(1 + v.numel(), device="cuda", dtype=torch.bfloat16)[1:].view(v.shape)
    odd.copy_(v)
    pad = torch.zeros(B, S, H, D + 4, device="cuda", dtype=torch.bfloat16)[..., 2:D + 2]
    pad.copy_(v)
    qs = torch.zeros(B * W, n_q, 2, Hq, D + 2, device="cuda", dtype=torch.bfloat16)[:, :, 1, :, 1:D + 1]
    qs.copy_(q)
    for kk, vv, qq in ((hm, v, q), (k, odd, q), (odd.clone().copy_(k), pad, qs), (hm, pad, qs)):
        o = torch.full((B * W, n_q, Hq, D + 6), 3.0, device="cuda", dtype=torch.bfloat16)
        got = x.attend(qq, kk, vv, i32(lens), out=o[..., 3:D + 3])
        _check(got, q, k, v, lens, W, sample=8)
        assert (o[..., :3] == 3).all() and (o[..., D + 3:] == 3).all()
    one = k[:1, :, :1].expand(B, S, H, D)                            # stride 0 in sentences and heads
    got = x.attend(q, one, one, i32(lens))
    _check(got, q, one, one, lens, W, sample=8)
    assert want.shape == q.shape and x.status() == 0
    x.close()


def test_extreme_scores():
    """One-hot weights, equal scores, and scores near fp32's end."""
    import verify_bs_step_gb300 as vbs
    B, W, Hq, S, D = 2, 1, 2, 100, 64
    for n_q in (1, 96):
        x = vbs.CrossAttention(B, W, Hq, D, max_q=n_q, max_len=S)
        q, k, v = _tensors(B, W, n_q, Hq, Hq, S, D, seed=4)
        for scale in (0.0, 30.0, -2.0, 1e-30):
            out = x.attend(q, k, v, i32([100, 63]), scale=scale)
            _check(out, q, k, v, [100, 63], W, scale=scale, sample=8)
        big = (q.float() * 2.0 ** 50).to(torch.bfloat16)
        out = x.attend(big, (k.float() * 2.0 ** 50).to(torch.bfloat16), v, i32([100, 63]), scale=1.0)
        s = torch.einsum("bqhd,bshd->bqhs", q.double(), k.double())
        s[1, :, :, 63:] = -float("inf")
        best = s.argmax(-1)
        want = torch.gather(v.permute(0, 2, 1, 3), 2, best.permute(0, 2, 1)[..., None].expand(-1, -1, -1, D))
        assert torch.equal(out, want.permute(0, 2, 1, 3))
        x.close()


def test_long_sources_are_split_and_joined():
    import verify_bs_step_gb300 as vbs
    for B, W, n_q, Hq, H, S, D in ((1, 1, 1, 4, 1, 30011, 128), (2, 4, 2, 2, 2, 6000, 64), (1, 1, 70, 1, 1, 9001, 64)):
        x = vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)
        for mul in (1.0, 6.0):
            q, k, v = _tensors(B, W, n_q, Hq, H, S, D, seed=8, mul=mul)
            lens = [S, 4097][:B]
            a = x.attend(q, k, v, i32(lens))
            _check(a, q, k, v, lens, W, sample=3)
            assert torch.equal(a, x.attend(q, k, v, i32(lens)))
        x.close()


def test_offsets_past_32_bits():
    import verify_bs_step_gb300 as vbs
    B, S, H, D = 3, 600000, 8, 128
    kv = torch.zeros(B, S, 2, H, D, device="cuda", dtype=torch.bfloat16)
    assert kv.stride(0) * (B - 1) > 1 << 31
    kv[:, :200] = torch.randn(B, 200, 2, H, D, device="cuda").to(torch.bfloat16)
    for n_q in (1, 70):
        q = torch.randn(B, n_q, H, D, device="cuda").to(torch.bfloat16)
        x = vbs.CrossAttention(B, 1, H, D, max_q=n_q, max_len=S)
        out = x.attend(q, kv[:, :, 0], kv[:, :, 1], i32([150, 7, 199]))
        _check(out, q, kv[:, :200, 0], kv[:, :200, 1], [150, 7, 199], 1, sample=4)
        hm = kv.view(B, S * 2 * H, D)[:, :S * H].view(B, H, S, D)     # head-major: head strides past 32 bits of bytes
        hm[:, :, :200] = torch.randn(B, H, 200, D, device="cuda").to(torch.bfloat16)
        t = hm.permute(0, 2, 1, 3)
        out = x.attend(q, t, t, i32([150, 7, 199]))
        _check(out, q, t[:, :200], t[:, :200], [150, 7, 199], 1, sample=4)
        x.close()
    del kv
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n_q", [1, 100])
def test_graph_replay_and_streams(n_q):
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _replay_and_streams(n_q, side)


def _replay_and_streams(n_q, own):
    import verify_bs_step_gb300 as vbs
    B, W, Hq, H, S, D = 2, 2, 4, 2, 120, 64
    x = vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)
    q, k, v = _tensors(B, W, n_q, Hq, H, S, D)
    lens = i32([120, 50])
    out = torch.zeros_like(q)
    x.attend(q, k, v, lens, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=own):
        x.attend(q, k, v, lens, out=out)
    q.copy_(_tensors(B, W, n_q, Hq, H, S, D, seed=9)[0])
    lens.copy_(i32([3, 119]))
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q, k, v, [3, 119], W, sample=8)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(3_000_000)
        q2 = q * 2
        got = x.attend(q2, k, v, lens) * 1
    side.synchronize()
    _check(got, q2, k, v, [3, 119], W, sample=8)
    x.close()


def test_refusals():
    import verify_bs_step_gb300 as vbs
    for kw in ({"heads": 3, "kv_heads": 2}, {"heads": 0}, {"W": 17}, {"W": 0}, {"D": 12}, {"D": 264}, {"D": 0},
               {"max_q": 0}, {"max_len": 0}, {"batch": 0}):
        a = {"batch": 1, "W": 1, "heads": 2, "D": 64, **kw}
        with pytest.raises(vbs.VbsError) as e:
            vbs.CrossAttention(**a)
        assert e.value.status == vbs.EINVAL
    x = vbs.CrossAttention(2, 2, 4, 64, kv_heads=2, max_q=3, max_len=10)
    q, k, v = _tensors(2, 2, 3, 4, 2, 10, 64)
    lens = i32([10, 4])
    for bad in (q[:3], q[:, :, :2], q.float(), q[..., :32], q.transpose(2, 3), q.cpu(), q[0]):
        with pytest.raises(ValueError):
            x.attend(bad, k, v, lens)
    for bad in (k[:1], k[:, :, :1], k.half(), k[:, :5]):
        with pytest.raises(ValueError):
            x.attend(q, bad, v, lens)
    for bad in (lens[:1], lens.long(), lens.cpu()):
        with pytest.raises(ValueError):
            x.attend(q, k, v, bad)
    many, kk, vv = _tensors(2, 2, 4, 4, 2, 11, 64)
    for args in ((many, k, v), (q, kk, vv)):                          # more tokens, more positions than announced
        with pytest.raises(vbs.VbsError) as e:
            x.attend(*args, lens)
        assert e.value.status == vbs.EINVAL
    with pytest.raises(vbs.VbsError):
        x.attend(q, k, v, lens, scale=float("nan"))
    x.attend(q, k, v, i32([11, -1]))
    assert x.status() == vbs.EINVAL and x.status() == 0
    none = x.attend(q, k[:, :0], v[:, :0], i32([0, 0]))              # no positions at all
    assert not none.any() and x.status() == 0
    x.close()
