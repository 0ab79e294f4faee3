"""Cross attention's tcgen05 tiles and its split kernel, each at shapes that reach it (the tests assert which one ran)."""

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


def _op(B, W, Hq, D, H, n_q, S):
    import verify_bs_step_gb300 as vbs
    return vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)


def _tensors(B, W, n_q, Hq, H, S, D, seed=0, mul=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(B * W, n_q, Hq, D, device="cuda", generator=g) * mul).to(torch.bfloat16)
    kv = torch.randn(B, S, 2, H, D, device="cuda", generator=g).to(torch.bfloat16)
    return q, kv[:, :, 0], kv[:, :, 1]


def _check(out, q, k, v, lens, W, scale=None, rows=None, sample=8):
    """Sampled tokens of every head of `rows` (all) against the oracle: one bf16 rounding a weight."""
    R, n_q, Hq, D = q.shape
    G = Hq // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    at = sorted({int(i) for i in np.linspace(0, n_q - 1, sample)})
    for r in range(R) if rows is None else rows:
        b, n = r // W, max(0, min(int(lens[r // W]), k.shape[1]))
        for h in range(Hq):
            check_rows(out[r, at, h].double().cpu(), q[r, at, h].double().cpu(), k[b, :n, h // G].double().cpu(),
                       v[b, :n, h // G].double().cpu(), [n] * len(at), scale, BF16, f"row {r} head {h}")


# head_dim up to 64 takes the tiles from 385 positions on, up to 128 from 257, whatever the rows past 16
S64, S128 = 450, 300


@pytest.mark.parametrize("W,n_q,Hq,H,S,D", [
    (1, 17, 1, 1, S64, 64), (1, 128, 2, 2, S64, 64), (1, 129, 2, 1, 512, 64), (1, 300, 2, 2, 385, 64),
    (3, 50, 4, 2, 768, 64), (16, 2, 2, 2, S64, 8), (2, 33, 3, 3, S64, 24), (1, 200, 2, 1, S64, 40),
    (1, 20, 2, 2, S128, 128), (1, 260, 2, 2, 257, 128), (2, 40, 6, 2, 640, 128), (5, 7, 4, 4, S128, 72),
    (1, 130, 2, 1, S128, 96), (1, 64, 2, 2, S128, 112),
])
def test_rows_and_head_dims(W, n_q, Hq, H, S, D):
    x = _op(4, W, Hq, D, H, n_q, S)
    q, k, v = _tensors(4, W, n_q, Hq, H, S, D, seed=D + n_q)
    for lens, scale in (([S, 65, 1, 0], None), ([0, S - 1, 64, S // 2], 0.9)):
        out = x.attend(q, k, v, i32(lens), scale=scale)
        assert x.tiles is True
        _check(out, q, k, v, lens, W, scale=scale)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("B,H,n_q,S,D", [(130, 8, 33, 400, 64), (130, 8, 33, 300, 128), (60, 4, 300, 400, 64),
                                         (60, 4, 300, 300, 96)])
def test_several_items_a_cta(B, H, n_q, S, D):
    """Several times as many (sentence, head, row tile) items as CTAs, empty and one-tile sentences among long ones."""
    x = _op(B, 1, H, D, H, n_q, S)
    q, k, v = _tensors(B, 1, n_q, H, H, S, D, seed=B + D)
    lens = [(0, 1, 63, 64, 65, S, 128, 0, S - 1, 200)[i % 10] for i in range(B)]
    lens = list(np.random.default_rng(B).permutation(lens))
    out = x.attend(q, k, v, i32(lens))
    assert x.tiles is True and B * H * -(-n_q // 128) > 608
    _check(out, q, k, v, lens, 1, rows=range(0, B, 3), sample=3)
    # every item, against the library's other order of the work: the sentences in reverse
    back = x.attend(q.flip(0), k.flip(0), v.flip(0), i32(lens[::-1]))
    assert torch.equal(back.flip(0), out)
    assert not out[torch.tensor([n == 0 for n in lens], device="cuda")].any() and x.status() == 0
    x.close()


@pytest.mark.parametrize("B", [1024, 1025, 1400])
def test_more_sentences_than_are_sorted(B):
    x = _op(B, 1, 1, 64, 1, 20, 400)
    q, k, v = _tensors(B, 1, 20, 1, 1, 400, 64, seed=B)
    lens = np.random.default_rng(B).integers(0, 401, size=B)
    out = x.attend(q, k, v, i32(lens))
    assert x.tiles is True
    _check(out, q, k, v, lens, 1, rows=range(0, B, 7), sample=2)
    assert x.status() == 0
    x.close()


@pytest.mark.parametrize("S,D", [(S64, 64), (S128, 128), (S128, 80)])
@pytest.mark.parametrize("n_q", [17, 150])
def test_what_lies_past_a_sentences_end_is_not_used(n_q, S, D):
    B, W, Hq, H = 4, 2, 4, 2
    x = _op(B, W, Hq, D, H, n_q, S)
    q, k, v = _tensors(B, W, n_q, Hq, H, S, D)
    lens = [S - 19, 0, 16, 64]
    clean = x.attend(q, k, v, i32(lens))
    assert x.tiles is True
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = float("nan"), float("inf")
        v[b, n::2] = float("nan")
        k[b, n::2] = -torch.finfo(torch.bfloat16).max
    out = x.attend(q, k, v, i32(lens))
    assert torch.equal(out, clean) and not out[2:4].any()
    _check(out, q, k, v, lens, W)
    x.close()


@pytest.mark.parametrize("S,D", [(S64, 64), (S128, 128), (S64, 40)])
def test_strides_and_layouts(S, D):
    """Head-major and interleaved K and V, each with the other; queries and outputs at odd offsets and strides; layouts
    that a tensor map cannot hold, which the split kernel takes."""
    B, W, Hq, H, n_q = 2, 3, 4, 2, 50
    x = _op(B, W, Hq, D, H, n_q, S)
    q, k, v = _tensors(B, W, n_q, Hq, H, S, D)
    lens = [S, S // 2 + 3]
    hk, hv = (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (k, v))
    pad = torch.zeros(B, S, H, D + 8, device="cuda", dtype=torch.bfloat16)[..., 8:]
    pad.copy_(v)
    odd = torch.empty(1 + v.numel(), device="cuda", dtype=torch.bfloat16)[1:].view(v.shape).copy_(v)
    qs = torch.zeros(B * W, n_q, 2, Hq, D + 2, device="cuda", dtype=torch.bfloat16)[:, :, 1, :, 1:D + 1]
    qs.copy_(q)
    heads = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)         # queries head-major
    for kk, vv, qq, tiles in ((hk, hv, q, True), (hk, v, qs, True), (k, hv, heads, True), (k, pad, qs, True),
                              (k, odd, q, False)):
        for lead, room in ((3, 6), (8, 16)):
            o = torch.full((B * W, n_q, Hq, D + room), 3.0, device="cuda", dtype=torch.bfloat16)
            got = x.attend(qq, kk, vv, i32(lens), out=o[..., lead:D + lead])
            assert x.tiles is tiles
            _check(got, q, k, v, lens, W, sample=4)
            assert (o[..., :lead] == 3).all() and (o[..., D + lead:] == 3).all()
    one = k[:1, :, :1].expand(B, S, H, D)                                  # stride 0 in sentences and heads
    _check(x.attend(q, one, one, i32(lens)), q, one, one, lens, W, sample=4)
    assert x.tiles is False and x.status() == 0
    x.close()


@pytest.mark.parametrize("S,D", [(S64, 64), (S128, 128)])
def test_extreme_scores(S, D):
    """Equal, reversed and one-hot weights; references past 65536; scores near fp32's end."""
    B, Hq, n_q = 2, 2, 140
    x = _op(B, 1, Hq, D, Hq, n_q, S)
    q, k, v = _tensors(B, 1, n_q, Hq, Hq, S, D, seed=4)
    lens = [S, 63]
    for scale in (0.0, 30.0, -2.0, 1e-30, -1e-30):
        out = x.attend(q, k, v, i32(lens), scale=scale)
        assert x.tiles is True
        _check(out, q, k, v, lens, 1, scale=scale)
    s = torch.einsum("bqhd,bshd->bqhs", q.double(), k.double())
    s[1, :, :, 63:] = -float("inf")
    for mul, sign in ((2.0 ** 10, 1), (2.0 ** 50, 1), (2.0 ** 10, -1)):    # scores of a million and of 1e31
        big, bigk = ((t.float() * mul).to(torch.bfloat16) for t in (q, k))
        out = x.attend(big, bigk, v, i32(lens), scale=float(sign))
        best = torch.where(s.isinf(), -float("inf"), s * sign).argmax(-1)
        want = torch.gather(v.permute(0, 2, 1, 3), 2, best.permute(0, 2, 1)[..., None].expand(-1, -1, -1, D))
        assert x.tiles is True and torch.equal(out, want.permute(0, 2, 1, 3))
    x.close()


@pytest.mark.parametrize("S,D", [(S64, 64), (S128, 128)])
def test_offsets_past_32_bits(S, D):
    """Sentences and heads more than 2^31 elements apart."""
    B, H, n_q = 3, 2, 40
    far = (1 << 31) + 512
    mem = torch.empty(far * 2 + far // 2 + S * 2 * D, device="cuda", dtype=torch.bfloat16)
    q, k, v = _tensors(B, 1, n_q, H, H, S, D, seed=2)
    lens = [S, 7, S - 1]
    x = _op(B, 1, H, D, H, n_q, S)
    for sent, head in ((far, D), (far, far // 2)):
        kk = mem.as_strided((B, S, H, D), (sent, 2 * D if head == D else D, head, 1))
        kk.copy_(k)
        out = x.attend(q, kk, v, i32(lens))
        assert x.tiles is True
        _check(out, q, k, v, lens, 1)
        out = x.attend(q, v, kk, i32(lens))
        _check(out, q, v, k, lens, 1)
    x.close()
    del mem, kk
    torch.cuda.empty_cache()


@pytest.mark.parametrize("S,D", [(S64, 64), (S128, 128)])
def test_graph_replay_and_streams(S, D):
    own = torch.cuda.Stream()
    with torch.cuda.stream(own):
        B, W, Hq, H, n_q = 2, 2, 4, 2, 100
        x = _op(B, W, Hq, D, H, n_q, S)
        q, k, v = _tensors(B, W, n_q, Hq, H, S, D)
        lens, out = i32([S, 50]), torch.zeros_like(q)
        x.attend(q, k, v, lens, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=own):
            x.attend(q, k, v, lens, out=out)
            x.attend(q, k, v, lens, out=out)
        q.copy_(_tensors(B, W, n_q, Hq, H, S, D, seed=9)[0])
        lens.copy_(i32([3, S - 1]))
        graph.replay()
        torch.cuda.synchronize()
        assert x.tiles is True
        _check(out, q, k, v, [3, S - 1], W)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(3_000_000)
        q2 = q * 2
        got = x.attend(q2, k, v, lens) * 1
    side.synchronize()
    _check(got, q2, k, v, [3, S - 1], W)
    x.close()


@pytest.mark.parametrize("S", [40, 900])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_split_kernel_keeps_16_bits_of_a_weight(S, D):
    """Two positions whose values all but cancel, so that a weight of 8 bits would show in the result: the weights are
    two bf16 parts, the second of them within half a step of what the first leaves (2^-8 of 2^-8)."""
    B, H = 16, 8
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.rand(B, 1, H, D, device="cuda", generator=g).to(torch.bfloat16)
    k, v = (torch.randn(B, S, H, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    k[:, :2] = (k[:, :2].float() / D).to(torch.bfloat16)                    # scores below 1
    s = torch.einsum("bhd,bshd->bhs", q[:, 0].double(), k[:, :2].double())
    ratio = torch.exp(s[..., 0] - s[..., 1])
    v[:, 1] = (-v[:, 0].double() * ratio[..., None]).to(torch.bfloat16)
    x = _op(B, 1, H, D, H, 1, S)
    out = x.attend(q, k, v, i32([2] * B), scale=1.0)
    assert x.tiles is False and x.status() == 0
    o, qq, kk, vv = (t.double().cpu() for t in (out[:, 0], q[:, 0], k[:, :2], v[:, :2]))
    for b in range(B):
        for h in range(H):
            check_rows(o[b, h:h + 1], qq[b, h:h + 1], kk[b, :, h], vv[b, :, h], [2], 1.0, BF16 * BF16, f"{b} {h}")
    x.close()


def test_which_kernel_ran():
    import ctypes

    import verify_bs_step_gb300 as vbs
    x = _op(1, 1, 1, 64, 1, 40, 500)
    assert x.tiles is None
    q, k, v = _tensors(1, 1, 40, 1, 1, 500, 64)
    x.attend(q, k, v, i32([500]))
    assert x.tiles is True
    x.attend(q[:, :1].contiguous(), k, v, i32([500]))
    assert x.tiles is False
    assert vbs.lib().xattn_kernel(None, ctypes.byref(ctypes.c_int())) == vbs.EINVAL
    assert vbs.lib().xattn_kernel(x.ctx, None) == vbs.EINVAL
    x.close()
