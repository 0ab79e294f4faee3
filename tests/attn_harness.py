"""Shared by the attention tests: the error bound, and a decode that fills a cache through the public calls."""

import numpy as np
import torch

from oracle import attn as oa

DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
BF16 = torch.finfo(torch.bfloat16).eps / 2          # a rounding to bf16, relative
FP16 = torch.finfo(torch.float16).eps / 2
FP32 = torch.finfo(torch.float32).eps / 2
# fp16 weights, the largest between 2^12 and 2^15: half the smallest fp16 step (2^-25) is 2^-37 of it at most, and a
# term is at most a code of QMAX in a scale below 2 / QMAX of the largest value
FP16_FLOOR = 2.0 ** -36


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def check_rows(got, q, k, v, seen, scale, weight_eps, what="", weight_floor=2.0 ** -125):
    """got [n, D] (bf16) against the fp64 attention of q [n, D] over k, v [T, D].

    The bound: the result's rounding; each weight's rounding (weight_eps) times sum p|v|; and the
    scores' own error, which moves every weight by that relative amount.  A score is an fp32 sum of
    D products of |q||k|, scaled (D + 4 roundings), and its power of two an approximation good
    to 2^-22 of a number up to |s| log2(e) (one rounding); sums of T weights in fp32 add T roundings.
    The score error and the sums' count twice, in the numerator and in the normalisation.
    A weight is held to weight_floor of the largest at best (where its format underflows).
    """
    got, q, k, v = (np.asarray(t, dtype=np.float64) for t in (got, q, k, v))
    want = oa.attention(q, k, v, seen, scale)
    size = oa.attention(q, k, np.abs(v), seen, scale)
    for i in range(q.shape[0]):
        t = max(0, min(int(seen[i]), k.shape[0]))
        if t == 0:
            assert not got[i].any(), f"{what}: query {i} sees nothing"
            continue
        mag = float((np.abs(k[:t]) @ np.abs(q[i])).max()) * abs(scale)
        score = (q.shape[1] + 8) * FP32 * mag * 1.5 + 2.0 ** -22
        bound = BF16 * np.abs(want[i]) + (weight_eps + 2 * score + 2 * t * FP32) * size[i] * (1 + BF16)
        bound = bound + t * weight_floor * np.abs(v).max()
        err = np.abs(got[i] - want[i])
        assert np.isfinite(got[i]).all(), f"{what}: query {i} is not finite"
        bad = err > bound
        assert not bad.any(), (f"{what}: query {i}, dim {int(np.argmax(err - bound))}: off by "
                               f"{err.max():.3e}, bound {bound[np.argmax(err - bound)]:.3e}")


class Decode:
    """A ragged decode on a PagedKV8: prompts, then positions written one by one with reorders between."""

    def __init__(self, fmt, lens, W, heads, H, D, block, gen, *, max_q=1, L=2, layer=1, seed=0, spread=0.7,
                 reorder_every=3, garbage=True, spare=0):
        import verify_bs_step_gb300 as vbs
        self.rng = np.random.default_rng(seed)
        self.lens, self.W, self.H, self.D, self.layer, self.spread = np.asarray(lens), W, H, D, layer, spread
        B = len(lens)
        self.R = B * W
        S = -(-max(lens) // block) + W * (gen // block + 3) + spare
        MB = (max(lens) + gen) // block + 1
        self.kv = kv = vbs.PagedKV8(B, W, L, H, D, heads=heads, max_q=max_q, blocks_per_sentence=S, max_blocks=MB,
                                    block=block, dtype=DT[fmt])
        if garbage:                                  # what no append has written: NaN in e4m3, -1 in int8
            kv.pool.view(torch.uint8).fill_(0xff)
            kv.scales.fill_(float("nan"))
        n = int(self.lens.sum())
        slots = kv.build(i32(lens), n)[0]
        kv.append(layer, *self.new(n), slots)
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
        def one():
            x = self.rng.standard_normal((n, self.H, self.D)) * np.exp(
                self.rng.standard_normal((n, self.H, 1)) * self.spread)
            return torch.from_numpy(x).to("cuda", torch.bfloat16)
        return one(), one()

    def rows(self):
        """Every row's cached K and V as held, [T, H, D] fp64 each."""
        out = []
        for r in range(self.R):
            cnt = np.zeros(self.R, dtype=np.int64)
            cnt[r] = self.ctx[r]
            slots = self.kv.slot_map(i32(np.zeros(self.R)), i32(cnt), int(cnt[r]))[0]
            k, v = self.kv.read(self.layer, slots)
            out.append((k.double().cpu().numpy(), v.double().cpu().numpy()))
        return out

    def check(self, out, q, ctx=None, scale=None, what=""):
        """out, q [R, n_q, heads, D] against the oracle, ctx cached positions a row."""
        ctx = self.ctx if ctx is None else np.asarray(ctx)
        scale = self.D ** -0.5 if scale is None else scale
        n_q, heads = q.shape[1], q.shape[2]
        G = heads // self.H
        o, qq = out.double().cpu().numpy(), q.double().cpu().numpy()
        for r, (k, v) in enumerate(self.rows()):
            seen = ctx[r] - n_q + 1 + np.arange(n_q)
            for h in range(heads):
                check_rows(o[r, :, h], qq[r, :, h], k[:, h // G], v[:, h // G], seen, scale, 2 * FP16,
                           f"{what} row {r} head {h}", FP16_FLOOR)
        assert self.kv.status() == 0
