"""A translation decode on the library's operators: ragged prompts, an 8-bit paged cache, beams, cross attention.

One decoder layer with random weights: every step writes the new token's K and V into the 8-bit cache, attends
to the row's past and to the sentence's encoder states, and takes one beam step that also remaps the cache.

    python examples/beam_decode.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import verify_bs_step_gb300 as vbs  # noqa: E402


class Decoder:
    def __init__(self, vocab=1000, heads=8, kv_heads=4, D=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        d = heads * D

        def weight(n, m):
            return (torch.randn(n, m, device="cuda", generator=g) / n ** 0.5).to(torch.bfloat16)
        self.vocab, self.heads, self.kv_heads, self.D = vocab, heads, kv_heads, D
        self.emb = torch.randn(vocab, d, device="cuda", generator=g).to(torch.bfloat16)
        self.wqkv = weight(d, (heads + 2 * kv_heads) * D)
        self.wo, self.wq2, self.wo2 = weight(d, d), weight(d, d), weight(d, d)
        self.wkv2 = weight(d, 2 * kv_heads * D)
        self.wout = weight(d, vocab)

    def qkv(self, x):
        y = (x @ self.wqkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.D)
        return y.split((self.heads, self.kv_heads, self.kv_heads), dim=1)


class Decode:
    """The decode of `batch` sentences x W beams: prompts (a list of token lists) and encoder states
    [batch, S, heads * D] with their lengths."""

    def __init__(self, model: Decoder, prompts, states, enc_len, *, W=4, steps=16, eos=2, block=16, dtype=torch.float8_e4m3fn):
        m, B = model, len(prompts)
        self.m, self.W, self.R, self.steps = m, W, B * W, steps
        longest = max(len(p) for p in prompts)
        self.kv = vbs.PagedKV8(B, W, 1, m.kv_heads, m.D, heads=m.heads, block=block, dtype=dtype,
                               blocks_per_sentence=-(-longest // block) + W * (-(-steps // block) + 2),
                               max_blocks=(longest + steps) // block + 1)
        self.cross = vbs.CrossAttention(B, W, m.heads, m.D, kv_heads=m.kv_heads, max_len=states.shape[1])
        self.bs = vbs.BeamSearch(B, W, m.vocab, eos=eos, max_len=steps, bos=1, pad=-1)
        self.enc_len = enc_len
        self.enc_k, self.enc_v = (states @ m.wkv2).view(B, -1, 2, m.kv_heads, m.D).unbind(2)
        # the prompts: tables and slots from their lengths, then their K and V
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        flat = torch.tensor([t for p in prompts for t in p], dtype=torch.int64, device="cuda")
        slots, _, _, _ = self.kv.build(lens, flat.numel())
        _, k, v = m.qkv(m.emb[flat])
        self.kv.append(0, k, v, slots)
        self.kv.prepare(0)
        self.start = lens.repeat_interleave(W)
        self.t = 0

    def step(self, observe=None):
        """One step; observe, if given, gets what its attention saw and gave before the cache is remapped."""
        m, kv, t = self.m, self.kv, self.t
        tok = self.bs.tokens if t else torch.ones(self.R, dtype=torch.int32, device="cuda")
        live = (tok >= 0).to(torch.int32)                       # rows of finished sentences write and see nothing
        x = m.emb[tok.clamp(min=0).long()]
        q, k, v = m.qkv(x)
        slots, _, _, _ = kv.slot_map(self.start + t, live, self.R)
        # the slot map lists the live rows' tokens one after the other
        kv.append(0, *self._listed(live, k, v), slots)
        ctx = (self.start + t + 1) * live
        kv.plan(ctx)
        a = kv.attend(0, q.unsqueeze(1)).view(self.R, -1)
        h = x + a @ m.wo
        q2 = (h @ m.wq2).view(self.R, 1, m.heads, m.D)
        c = self.cross.attend(q2, self.enc_k, self.enc_v, self.enc_len).view(self.R, -1)
        logits = (h + c @ m.wo2) @ m.wout
        if observe is not None:
            observe({"q": q, "ctx": ctx, "self": a, "q2": q2, "cross": c})
        self.bs.step_paged(logits, kv, t + 1)
        kv.copy()
        self.t += 1

    def _listed(self, live, k, v):
        order = torch.argsort(live, descending=True, stable=True)
        return k[order], v[order]

    def run(self):
        while self.t < self.steps:
            self.step()
        return self.bs.finalize()

    def close(self):
        for c in (self.kv, self.cross, self.bs):
            c.close()


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    model = Decoder()
    prompts = [[(7 * i + j) % model.vocab for j in range(n)] for i, n in enumerate((1, 37, 5, 64))]
    states = torch.randn(4, 50, model.heads * model.D, device="cuda", generator=g).to(torch.bfloat16)
    d = Decode(model, prompts, states, torch.tensor([50, 12, 33, 1], dtype=torch.int32, device="cuda"))
    seqs, lens, scores = d.run()
    assert d.kv.status() == 0 and d.cross.status() == 0 and d.bs.status() == 0
    for s, n, x in zip(seqs.tolist(), lens.tolist(), scores.tolist()):
        print(f"{x:9.4f}  {s[:n]}")
    d.close()


if __name__ == "__main__":
    main()
