"""Infinities and NaN of V that a row sees: their product with the weight as held in fp32, in every kernel alike.

A weight is positive for a finite score, so that an infinity stays one; it is 0 for a score of -inf, which makes NaN of an
infinity.  A weight that is too small for fp32 may count as either, but the element is never left out."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, check_rows, i32
from tests.test_gpu_prompt import filled, starts, tensors

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


# how a prompt is brought to each form: items of one row tile, of two, and rows 2 bytes off for the other kernel
def prompts(form, D):
    import verify_bs_step_gb300 as vbs
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return (filled(vbs, 2 * 64 * (sms + 1)) if form == "two" else vbs.PromptAttention)(2, D, kv_heads=1)


def shifted(x):
    flat = torch.empty(x.numel() + 1, device="cuda", dtype=x.dtype)[1:].view(x.shape)
    return flat.copy_(x)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("form,D", [("one", 64), ("one", 128), ("one", 136), ("two", 64), ("two", 128), ("rows", 64)])
def test_prompts(form, D, causal):
    x = prompts(form, D)
    n = 20
    cu = starts([n, 300])
    q, k, v = tensors(n + 300, 2, 1, D)
    q[..., 0] = q[..., 0].abs() + 0.5
    k[:7, 0, 0] = -INF                               # request 0's first seven positions have no weight
    k[9, 0, 0], k[11, 0, 0] = -3e3 * D ** 0.5, -3e3 * D ** 0.5   # and these less than fp32 holds
    v[3, 0, 5], v[4, 0, 6], v[5, 0, 7] = INF, -INF, NAN
    v[9, 0, 8], v[11, 0, 9] = INF, -INF
    v[14, 0, 10], v[15, 0, 11] = INF, -INF           # these have some
    if form == "rows":
        q, k, v = shifted(q), shifted(k), shifted(v)
    out = x.attend(q, k, v, i32(cu), causal=causal)
    assert x.tiles is (form != "rows")
    see = np.arange(n)[:, None] >= np.arange(n)[None] if causal else np.ones((n, n), dtype=bool)   # token, position
    none = ~see[:, 7:].any(1)                        # all that these see scores -inf
    assert out[:n][none].isnan().all() and torch.isfinite(out[n:]).all()
    some = torch.tensor(~none)
    for p, d, z in ((3, 5, NAN), (4, 6, NAN), (5, 7, NAN), (14, 10, INF), (15, 11, -INF)):
        at = torch.tensor(see[:, p]) & some
        got = out[:n][at][..., d]
        assert (got.isnan() if z != z else got == z).all(), (p, d)
        assert torch.isfinite(out[:n][some & ~at][..., d]).all(), (p, d)
    for p, d in ((9, 8), (11, 9)):
        at = torch.tensor(see[:, p]) & some
        assert not torch.isfinite(out[:n][at][..., d]).any() and torch.isfinite(out[:n][some & ~at][..., d]).all(), (p, d)
    # all else is the attention of the positions that have weight
    o, qq, kk, vv = (t.double().cpu().numpy() for t in (out, q, k, v))
    o[..., 5:12] = vv[..., 5:12] = 0
    for t in np.flatnonzero(~none):
        live = np.flatnonzero(see[t] & (kk[:n, 0, 0] > -100))
        for h in range(2):
            check_rows(o[t:t + 1, h], qq[t:t + 1, h], kk[live, 0], vv[live, 0], [len(live)], D ** -0.5, BF16,
                       f"token {t} head {h}")
    assert x.status() == 0
    x.close()


def cache(lens, W, n_q, heads, H, D, spare=0):
    from tests.test_gpu_attn16 import Decode16
    d = Decode16(lens, W, heads, H, D, 16, 0, max_q=n_q, seed=D, spare=spare)
    q = d.q(n_q, heads)
    q[..., 0] = q[..., 0].abs() + 0.5
    d.kv.plan(i32(d.ctx), n_q)
    pages = d.kv.table()[0].tolist()                 # sentence 0's, which all its beams share

    def cell(side, p, dim):                          # of K/V head 0
        return (pages[p // 16], d.layer, side, 0, p % 16, dim)
    return d, q, cell


def seen(out, n_q, W, G, p, length):
    """Which rows of out [R, n_q, heads] read position p of sentence 0 through K/V head 0."""
    m = torch.zeros(out.shape[:3], dtype=torch.bool)
    for i in range(n_q):
        m[:W, i, :G] = p < length - n_q + 1 + i
    return m


PAGED = [(1, 1, 64, 4, 2), (4, 1, 128, 4, 2), (1, 4, 80, 4, 1), (1, 8, 128, 8, 2), (3, 2, 64, 8, 2), (2, 8, 96, 4, 2), (1, 2, 256, 4, 2),
         (1, 12, 256, 4, 2)]                         # W, n_q, D, heads, H


@pytest.mark.parametrize("spare", [0, 900])         # segments whole and in pieces
@pytest.mark.parametrize("W,n_q,D,heads,H", PAGED)
def test_cache_however_small_the_weight_it_is_not_left_out(W, n_q, D, heads, H, spare):
    """Also where such a position is all that a warp or a piece of the line has seen."""
    length = 33                                      # position 32 stands in a unit of its own
    d, q, cell = cache([length, 90], W, n_q, heads, H, D, spare)
    want = d.kv.attend(d.layer, q)
    G = heads // H
    for p in (0, 15, 16, 20, 32):
        k_at, v_at = cell(0, p, 0), cell(1, p, 5)
        old = d.kv.pool[k_at].clone(), d.kv.pool[v_at].clone()
        d.kv.pool[k_at] = -3e3 * D ** 0.5
        clean = d.kv.attend(d.layer, q)
        assert torch.isfinite(clean).all()
        d.kv.pool[v_at] = INF
        out = d.kv.attend(d.layer, q)
        m = torch.zeros(out.shape, dtype=torch.bool)
        m[..., 5] = seen(out, n_q, W, G, p, length)
        assert not torch.isfinite(out[m]).any(), (p, out[m])
        assert torch.equal(out[~m], clean[~m]), p
        d.kv.pool[k_at], d.kv.pool[v_at] = old
    assert torch.equal(d.kv.attend(d.layer, q), want) and d.kv.status() == 0
    d.kv.close()


@pytest.mark.parametrize("spare", [0, 900])
@pytest.mark.parametrize("W,n_q,D,heads,H", PAGED)
def test_cache_a_position_without_weight_makes_nan_of_an_infinity(W, n_q, D, heads, H, spare):
    length = 33                                      # position 32 stands in a unit of its own
    d, q, cell = cache([length, 90], W, n_q, heads, H, D, spare)
    want = d.kv.attend(d.layer, q)
    G = heads // H
    for p in (0, 15, 16, 20, 32):
        k_at, v_at = cell(0, p, 0), cell(1, p, 5)
        old = d.kv.pool[k_at].clone(), d.kv.pool[v_at].clone()
        d.kv.pool[k_at] = -INF
        clean = d.kv.attend(d.layer, q)
        assert torch.isfinite(clean).all()
        d.kv.pool[v_at] = INF
        out = d.kv.attend(d.layer, q)
        m = torch.zeros(out.shape, dtype=torch.bool)
        m[..., 5] = seen(out, n_q, W, G, p, length)
        assert out[m].isnan().all(), (p, out[m])
        assert torch.equal(out[~m], clean[~m]), p
        d.kv.pool[k_at], d.kv.pool[v_at] = old
    assert torch.equal(d.kv.attend(d.layer, q), want) and d.kv.status() == 0
    d.kv.close()


@pytest.mark.parametrize("spare", [0, 900])         # segments whole and in pieces
@pytest.mark.parametrize("W,n_q,D,heads,H", PAGED)
def test_cache_an_infinity_that_has_weight_stays_one(W, n_q, D, heads, H, spare):
    length = 150
    d, q, cell = cache([length, 90], W, n_q, heads, H, D, spare)
    want = d.kv.attend(d.layer, q)
    d.check(want, q)
    for p in (0, 1, 7, 15, 16, 40, 63, 64, 100, 129, 143, 144, length - n_q, length - 1):
        for dim, z in ((5, INF), (D - 1, -INF)):
            at = cell(1, p, dim)
            old = d.kv.pool[at].clone()
            d.kv.pool[at] = z
            out = d.kv.attend(d.layer, q)
            m = torch.zeros(out.shape, dtype=torch.bool)
            m[..., dim] = seen(out, n_q, W, heads // H, p, length)
            assert (out[m] == z).all(), (p, dim, out[m])
            assert torch.equal(out[~m], want[~m]), (p, dim)
            d.kv.pool[at] = old
    assert d.kv.status() == 0
    d.kv.close()




@pytest.mark.parametrize("G", [1, 4])
def test_prompts_a_nan_costs_no_more_than_a_few_times_the_call(G):
    """One that a request of many tokens shares an item with, and ones among its own, near and far: looking for them takes a
    few times what the attention does (it took some hundred times that, and with the tokens came near the limit of waits)."""
    import verify_bs_step_gb300 as vbs
    n, D = 30000, 128
    cu = i32(starts([100, n]))
    q, k, v = tensors(100 + n, G, 1, D)
    x = vbs.PromptAttention(G, D, kv_heads=1)

    def ms():
        best = 1e9
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            x.attend(q, k, v, cu, causal=False, out=out)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    out = torch.empty(100 + n, G, D, device="cuda", dtype=torch.bfloat16)
    clean = ms()
    want = out.clone()
    v = v.clone()
    v[50, 0, 5] = NAN
    one = ms()
    assert out[:100, :, 5].isnan().all()
    out[:100, :, 5] = want[:100, :, 5]
    assert torch.equal(out, want)
    for p in (103, 17000, 99 + n):
        v[p, 0, 7] = INF
    several = ms()
    assert (out[100:, :, 7] == INF).all()
    out[:100, :, 5], out[100:, :, 7] = want[:100, :, 5], want[100:, :, 7]
    assert torch.equal(out, want) and x.status() == 0
    v[100:] = NAN                                    # all that the request has
    all_ = ms()
    print(f"{clean:.3f} ms, with one NaN {one:.3f}, several infinities {several:.3f}, all NaN {all_:.3f}")
    assert out[100:].isnan().all()
    assert max(one, several) < 20 * clean and all_ < 100 * clean, (clean, one, several, all_)
    x.close()
