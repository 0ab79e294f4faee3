"""Attention over the 16-bit paged cache against the fp64 oracle: weights of 16 bits, one rounding of the result."""

import numpy as np
import pytest
import torch

from tests.attn_harness import BF16, check_rows, i32

pytestmark = pytest.mark.gpu



def weight_eps(rows, D):
    """One rounding to bf16, or, for up to 16 rows that share a K/V head or head_dim above 128, two parts: what the second
    one's rounding leaves."""
    return BF16 if rows > 16 and D <= 128 else BF16 * BF16 * 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


class Decode16:
    """A ragged decode on a PagedKV16: prompts, then positions written one by one with reorders between.  What no
    append has written is NaN."""

    def __init__(self, lens, W, heads, H, D, block, gen, *, max_q=1, L=2, layer=1, seed=0, reorder_every=3, spare=0):
        import verify_bs_step_gb300 as vbs
        self.rng = np.random.default_rng(seed)
        self.lens, self.W, self.H, self.D, self.layer, self.block = np.asarray(lens), W, H, D, layer, block
        B = len(lens)
        self.R = B * W
        S = -(-max(lens) // block) + W * (gen // block + 3) + spare
        MB = (max(lens) + gen) // block + 1
        self.kv = kv = vbs.PagedKV16(B, W, L, H, D, heads=heads, max_q=max_q, blocks_per_sentence=S, max_blocks=MB, block=block)
        kv.pool.fill_(float("nan"))
        n = int(self.lens.sum())
        kv.append(layer, *self.new(n), kv.build(i32(lens), n)[0])
        for t in range(gen):
            if t and t % reorder_every == 0:
                par = np.sort(self.rng.integers(0, W, size=(B, W)))
                kv.reorder(i32((par + np.arange(B)[:, None] * W).reshape(-1)), t)
            else:
                kv.prepare(t)
            at = np.repeat(self.lens + t, W)
            kv.append(layer, *self.new(self.R), kv.slot_map(i32(at), i32([1] * self.R), self.R)[0])
        self.ctx = np.repeat(self.lens + gen, W)
        assert kv.status() == 0

    def new(self, n):
        return tuple(torch.from_numpy(self.rng.standard_normal((n, self.H, self.D))).to("cuda", torch.bfloat16) for _ in range(2))

    def q(self, n_q, heads, mul=1.0):
        return torch.from_numpy(self.rng.standard_normal((self.R, n_q, heads, self.D)) * mul).to("cuda", torch.bfloat16)

    def rows(self):
        """Every row's cached K and V, [T, H, D] fp64 each."""
        table, out = self.kv.table().cpu().numpy(), []
        pool = self.kv.pool[:, self.layer]
        for r in range(self.R):
            p = np.arange(self.ctx[r])
            x = pool[torch.tensor(table[r][p // self.block], device="cuda").long()][
                torch.arange(len(p), device="cuda"), :, :, torch.tensor(p % self.block, device="cuda")]
            out.append(x.double().cpu().numpy().transpose(1, 0, 2, 3))
        return out

    def check(self, out, q, ctx=None, scale=None, what=""):
        ctx = self.ctx if ctx is None else np.asarray(ctx)
        scale = self.D ** -0.5 if scale is None else scale
        n_q, heads = q.shape[1], q.shape[2]
        G = heads // self.H
        o, qq = out.double().cpu().numpy(), q.double().cpu().numpy()
        for r, (k, v) in enumerate(self.rows()):
            for h in range(heads):
                check_rows(o[r, :, h], qq[r, :, h], k[:, h // G], v[:, h // G], ctx[r] - n_q + 1 + np.arange(n_q), scale,
                           weight_eps(self.W * n_q * G, self.D), f"{what} row {r} head {h}")
        assert self.kv.status() == 0


@pytest.mark.parametrize("spare", [0, 900])         # segments whole and in pieces
@pytest.mark.parametrize("lens,W,n_q,heads,H,D,block,gen", [
    ([1], 1, 1, 1, 1, 8, 16, 0), ([37, 0, 5], 4, 1, 8, 2, 64, 16, 9), ([130], 5, 1, 4, 4, 128, 8, 20), ([70, 3], 2, 1, 16, 1, 128, 24, 5),
    ([33, 64], 1, 8, 8, 2, 128, 32, 0), ([20], 1, 32, 6, 3, 80, 16, 0), ([9, 100, 31], 16, 1, 2, 1, 40, 16, 6), ([50], 2, 3, 2, 2, 256, 16, 4),
    ([300, 2], 1, 1, 4, 4, 96, 64, 0), ([400], 1, 5, 8, 1, 256, 16, 0), ([17, 18], 3, 4, 5, 1, 64, 1, 3)])
def test_matches_the_oracle(lens, W, n_q, heads, H, D, block, gen, spare):
    d = Decode16(lens, W, heads, H, D, block, gen, max_q=n_q, seed=D, spare=spare)
    q = d.q(n_q, heads)
    d.kv.plan(i32(d.ctx), n_q)
    d.check(d.kv.attend(d.layer, q), q)
    d.check(d.kv.attend(d.layer, q * 4, scale=-0.8), q * 4, scale=-0.8)
    ctx = np.maximum(0, d.ctx - np.arange(d.R) * 7 - 1)          # shorter contexts, some of them empty
    d.kv.plan(i32(ctx), n_q)
    d.check(d.kv.attend(d.layer, q), q, ctx=ctx)
    d.kv.close()


@pytest.mark.parametrize("spare", [0, 900])
@pytest.mark.parametrize("n_q,W,D,heads", [(1, 3, 64, 4), (4, 2, 128, 4), (8, 1, 80, 8), (1, 2, 256, 2)])
def test_infinities_and_nan_reach_only_those_who_see_them(n_q, W, D, heads, spare):
    """A beam's own page that holds them leaves the other beams as they are, a later token's the earlier tokens."""
    d = Decode16([41, 90], W, heads, 2, D, 16, 6 if W > 1 else 0, max_q=n_q, spare=spare, reorder_every=100)
    q = d.q(n_q, heads)
    d.kv.plan(i32(d.ctx), n_q)
    want = d.kv.attend(d.layer, q)
    d.check(want, q)
    table = d.kv.table().cpu().numpy()
    # row 0's last two positions (a page of its own, or the step's last tokens) hold what is not finite
    for back, (side, z) in ((1, (1, float("inf"))), (2, (1, float("nan")))):
        p = int(d.ctx[0]) - back
        d.kv.pool[int(table[0][p // 16]), d.layer, side, 0, p % 16, 3 * back] = z
    out = d.kv.attend(d.layer, q)
    G = heads // 2
    hit = torch.zeros_like(out, dtype=torch.bool)
    for back in (1, 2):
        for i in range(n_q):
            if n_q - 1 - i < back:
                hit[0, i, :G, 3 * back] = True
    assert out[hit].isfinite().sum() == 0 and torch.isfinite(out[~hit]).all()
    assert (out[0, n_q - 1, :G, 3] == float("inf")).all() and out[0, n_q - 1, :G, 6].isnan().all()
    assert torch.equal(out[~hit], want[~hit])
    # a key that is not finite in a page of row 0's own
    p = int(d.ctx[0]) - 1
    d.kv.pool[int(table[0][p // 16]), d.layer, 0, 1, p % 16, 0] = float("nan")
    out = d.kv.attend(d.layer, q)
    assert out[0, n_q - 1, G:].isnan().all()
    assert torch.equal(out[1:, :, G:], want[1:, :, G:]) and torch.equal(out[0, :n_q - 1, G:], want[0, :n_q - 1, G:])
    d.kv.close()


def test_a_plan_does_not_outlive_its_tables():
    import verify_bs_step_gb300 as vbs
    kv = vbs.PagedKV16(1, 2, 1, 1, 16, heads=1, blocks_per_sentence=8, max_blocks=4, block=4)
    q = torch.ones(2, 1, 1, 16, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(vbs.VbsError):
        kv.attend(0, q)                              # not planned yet
    x = torch.ones(3, 1, 16, device="cuda")
    kv.append(0, x, x, kv.build(i32([3]), 3)[0])
    for change in (lambda: kv.prepare(0), lambda: kv.reorder(i32([0, 1]), 1), lambda: kv.prefill(3), lambda: kv.build(i32([3]))):
        kv.plan(i32([3, 3]))
        kv.attend(0, q)
        change()
        with pytest.raises(vbs.VbsError) as e:
            kv.attend(0, q)
        assert e.value.status == vbs.ESTATE
    kv.plan(i32([3, 9]))                             # more than the row's table covers: held to it, and told
    kv.attend(0, q)
    assert kv.status() == vbs.EINVAL
    bs = vbs.BeamSearch(1, 2, 20, max_len=4)
    kv.prepare(0)
    bs.step_paged(torch.randn(2, 20, device="cuda").to(torch.bfloat16), kv, 1)
    for f in (lambda: kv.plan(i32([3, 3])), lambda: kv.append(0, x, x, torch.arange(3, device="cuda"))):
        with pytest.raises(vbs.VbsError) as e:       # copies pending
            f()
        assert e.value.status == vbs.ESTATE
    kv.copy()
    kv.plan(i32([4, 4]))
    kv.attend(0, q)
    kv.close()
    bs.close()


def test_strided_queries_streams_and_graphs():
    d = Decode16([70, 33], 2, 4, 2, 64, 16, 5)
    q = d.q(1, 4)
    d.kv.plan(i32(d.ctx))
    want = d.kv.attend(d.layer, q)
    d.check(want, q)
    wide = torch.full((4, 1, 6, 67), 7.0, device="cuda", dtype=torch.bfloat16)
    wide[:, :, 1:5, 1:65] = q
    out = torch.full_like(wide, 5.0)
    d.kv.attend(d.layer, wide[:, :, 1:5, 1:65], out=out[:, :, :4, 3:])
    assert torch.equal(out[:, :, :4, 3:], want) and (out[:, :, 4:] == 5).all() and (out[..., :3] == 5).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = d.kv.attend(d.layer, q)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    d.kv.close()


def test_a_long_row_past_32_bits():
    """A pool of more than 2^31 elements, its last pages read and written."""
    import verify_bs_step_gb300 as vbs
    H, D, block = 8, 128, 64
    S, n = 8500, 2100                                # 2 x 8500 x 2 x 8 x 64 x 128 = 2.2e9 elements
    kv = vbs.PagedKV16(2, 1, 1, H, D, heads=H, blocks_per_sentence=S, max_blocks=40, block=block,
                       pool=torch.empty(2 * S, 1, 2, H, block, D, device="cuda", dtype=torch.bfloat16))
    slots = kv.build(i32([0, n]), n)[0]
    # sentence 1's table names its first pages: let it name its last ones (views() shows the library's own memory)
    pages = -(-n // block)
    kv.views()[0][1, :pages] += S - pages
    slots = slots + (S - pages) * block
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(n, H, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    kv.append(0, k, v, slots)
    q = torch.randn(2, 1, H, D, device="cuda", generator=g).to(torch.bfloat16)
    kv.plan(i32([0, n]))
    out = kv.attend(0, q)
    assert not out[0].any()
    for h in range(H):
        check_rows(out[1, :, h].double().cpu(), q[1, :, h].double().cpu(), k[:, h].double().cpu(), v[:, h].double().cpu(), [n],
                   D ** -0.5, weight_eps(1, D), f"head {h}")
    assert kv.status() == 0
    kv.close()


def test_refusals():
    import verify_bs_step_gb300 as vbs
    kv = vbs.PagedKV16(1, 2, 1, 1, 16, heads=2, blocks_per_sentence=8, max_blocks=4, block=4, max_q=2)
    kv.build(i32([3]))
    kv.plan(i32([3, 3]))
    q = torch.ones(2, 1, 2, 16, device="cuda", dtype=torch.bfloat16)
    kv.attend(0, q)
    bad = [lambda: kv.plan(i32([3])), lambda: kv.plan(i32([3, 3]).long()), lambda: kv.plan(i32([3, 3]), 3), lambda: kv.plan(i32([3, 3]), 0),
           lambda: kv.plan(i32([3, 3]).cpu()), lambda: kv.attend(1, q), lambda: kv.attend(0, q[:1]), lambda: kv.attend(0, q.float()),
           lambda: kv.attend(0, q, scale=float("inf")), lambda: kv.attend(0, q.cpu()), lambda: kv.attend(0, q, out=q[:, :, :1])]
    for f in bad:
        with pytest.raises((ValueError, vbs.VbsError)):
            f()
    kv.close()
