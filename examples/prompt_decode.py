"""A decoder-only beam decode on the library's operators: packed prompts, rotary positions, a 16-bit paged cache, beams.

Two decoder layers with random weights: the prompts go through the layers packed one after the other (rotary positions
and the cache write in one call, then attention of each prompt to itself); every step rotates and writes the new token's
rows, attends to the row's past over the cache, and takes one beam step that also remaps it.

    python examples/prompt_decode.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import verify_bs_step_gb300 as vbs  # noqa: E402


class Decoder:
    def __init__(self, vocab=1000, layers=2, heads=8, kv_heads=2, D=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        d = heads * D

        def weight(n, m):
            return (torch.randn(n, m, device="cuda", generator=g) / n ** 0.5).to(torch.bfloat16)
        self.vocab, self.layers, self.heads, self.kv_heads, self.D = vocab, layers, heads, kv_heads, D
        self.emb = torch.randn(vocab, d, device="cuda", generator=g).to(torch.bfloat16)
        self.wqkv = [weight(d, (heads + 2 * kv_heads) * D) for _ in range(layers)]
        self.wo = [weight(d, d) for _ in range(layers)]
        self.wout = weight(d, vocab)
        self.rotary = vbs.Rotary(D, base=10000.0, scaling="parts", factor=4.0, original=4096)

    def qkv(self, layer, x):
        """Queries, keys and values of tokens x [N, heads * D]: three slices of one product."""
        y = (x @ self.wqkv[layer]).view(x.shape[0], self.heads + 2 * self.kv_heads, self.D)
        return y.split((self.heads, self.kv_heads, self.kv_heads), dim=1)


class Decode:
    """The decode of `batch` sentences x W beams after `prompts` (a list of token lists, none empty)."""

    def __init__(self, model: Decoder, prompts, *, W=4, steps=16, eos=2, block=16, observe=None):
        m, B = model, len(prompts)
        self.m, self.W, self.R, self.steps = m, W, B * W, steps
        longest = max(len(p) for p in prompts)
        self.kv = vbs.PagedKV16(B, W, m.layers, m.kv_heads, m.D, heads=m.heads, block=block,
                                blocks_per_sentence=-(-longest // block) + W * (-(-steps // block) + 2),
                                max_blocks=(longest + steps) // block + 1)
        self.prompt = vbs.PromptAttention(m.heads, m.D, kv_heads=m.kv_heads)
        self.bs = vbs.BeamSearch(B, W, m.vocab, eos=eos, max_len=steps, bos=1, pad=-1)
        # the prompts, all tokens of all sentences at once
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        flat = torch.tensor([t for p in prompts for t in p], dtype=torch.int64, device="cuda")
        slots, pos, _, cu = self.kv.build(lens, flat.numel())
        x = m.emb[flat]
        for layer in range(m.layers):
            q, k, v = m.qkv(layer, x)
            # rotated in place: the prompts' attention reads what the cache holds
            self.kv.append(layer, k, v, slots, rotary=m.rotary, pos=pos, q=q, q_out=q, k_out=k)
            a = self.prompt.attend(q, k, v, cu)
            if observe is not None:
                observe({"layer": layer, "q": q, "k": k, "v": v, "cu": cu, "out": a})
            x = x + a.view(len(flat), -1) @ m.wo[layer]
        self.kv.prepare(0)
        self.start = lens.repeat_interleave(W)
        self.first = x[cu[1:].long() - 1].repeat_interleave(W, 0)     # the prompts' last tokens, for the first step
        self.t = 0

    def step(self, observe=None):
        """One step; observe, if given, gets what each layer's attention saw and gave before the cache is remapped."""
        m, kv, t = self.m, self.kv, self.t
        if t == 0:
            x = self.first                                        # their attention was the prompts'
        else:
            live = (self.bs.tokens >= 0).to(torch.int32)          # rows of finished sentences write and see nothing
            x = m.emb[self.bs.tokens.clamp(min=0).long()]
            slots, _, rows, _ = kv.slot_map(self.start + (t - 1), live, self.R)
            # the slot map lists the live rows one after the other: back to a slot a row, -1 for the others
            at = torch.cumsum(live, 0) - 1
            slots = torch.where(live > 0, slots[at.clamp(min=0)], -1)
            pos = torch.where(live > 0, self.start + (t - 1), -1).to(torch.int32)
            kv.plan((self.start + t) * live)
            for layer in range(m.layers):
                q, k, v = m.qkv(layer, x)
                q = q.contiguous()
                kv.append(layer, k, v, slots, rotary=m.rotary, pos=pos, q=q, q_out=q)
                a = kv.attend(layer, q.unsqueeze(1))
                if observe is not None:
                    observe({"layer": layer, "q": q, "ctx": (self.start + t) * live, "out": a})
                x = x + a.view(self.R, -1) @ m.wo[layer]
        self.bs.step_paged(x @ m.wout, kv, t)
        kv.copy()
        self.t += 1

    def run(self):
        while self.t < self.steps:
            self.step()
        return self.bs.finalize()

    def close(self):
        for c in (self.kv, self.prompt, self.bs):
            c.close()


def main():
    model = Decoder()
    prompts = [[(7 * i + j) % model.vocab for j in range(n)] for i, n in enumerate((1, 37, 5, 200))]
    d = Decode(model, prompts)
    seqs, lens, scores = d.run()
    assert d.kv.status() == 0 and d.prompt.status() == 0 and d.bs.status() == 0
    for s, n, x in zip(seqs.tolist(), lens.tolist(), scores.tolist()):
        print(f"{x:9.4f}  {s[:n]}")
    d.close()


if __name__ == "__main__":
    main()
