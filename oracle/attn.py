"""Block tables, the paged cache in 8 and 16 bits, attention over it, over an encoder's states and of prompts, rotary
positions.

TEST INFRASTRUCTURE.  Plain loops in fp64 (numpy); shares no code with the CUDA library.

What each function states:

* ``build_tables`` / ``slot_map``: requests of given lengths get consecutive blocks of their own;
  token p of a row lives in slot table[row][p // block] * block + p % block.
* ``scale_exponent`` / ``quantise``: one power-of-two scale per page and head, the smallest that
  holds the page's largest magnitude, and codes rounded to nearest, ties to even.
* ``append``: tokens written into pages in order; a page continued past its first slot never
  lowers its scale, and when the scale grows the codes already there are rounded again.
* ``rotate``: a pair (a, b) of dims at position p becomes amp (a cos pf - b sin pf, b cos pf + a sin pf).
* ``frequencies``: radians a position of each pair, scaled for long contexts.
* ``attention``: softmax(scale q k^T) v over the positions a query sees; zeros where it sees none.
"""

from __future__ import annotations

import math

import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}
E_LO, E_HI = -60, 60


def build_tables(lens, W: int, S: int, MB: int, block: int):
    B = len(lens)
    table = np.full((B * W, MB), -1, dtype=np.int32)
    nblk = np.zeros(B * W, dtype=np.int32)
    refcnt = np.zeros(B * S, dtype=np.int32)
    stack = np.zeros(B * S, dtype=np.int32)
    top = np.zeros(B, dtype=np.int32)
    for b, n in enumerate(lens):
        pages = -(-int(n) // block)
        table[b * W:(b + 1) * W, :pages] = b * S + np.arange(pages)
        nblk[b * W:(b + 1) * W] = pages
        refcnt[b * S:b * S + pages] = W
        stack[b * S:(b + 1) * S] = b * S + S - 1 - np.arange(S)
        top[b] = S - pages
    return table, nblk, refcnt, stack, top


def slot_map(table, rows, start, count, block: int, cap: int):
    """(slots, pos, row, cu) of the requests' tokens, -1 past the last one."""
    slots, pos, row = (np.full(cap, -1, dtype=np.int64) for _ in range(3))
    cu = np.zeros(len(rows) + 1, dtype=np.int64)
    o = 0
    for i, r in enumerate(rows):
        for p in range(int(start[i]), int(start[i]) + int(count[i])):
            slots[o] = int(table[r][p // block]) * block + p % block
            pos[o], row[o] = p, r
            o += 1
        cu[i + 1] = o
    return slots, pos, row, cu


def scale_exponent(amax: float, fmt: str) -> int:
    """The smallest e in [E_LO, E_HI] with amax <= QMAX 2^e (E_HI if there is none)."""
    if amax <= 0:
        return E_LO
    e = math.floor(math.log2(amax / QMAX[fmt])) - 1
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    return max(E_LO, min(E_HI, e))


def quantise(x, fmt: str):
    """The codes' numbers nearest to x (ties to even, magnitudes held at QMAX), in fp64."""
    x = np.clip(np.asarray(x, dtype=np.float64), -QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return np.round(x)
    _, ex = np.frexp(x)
    ulp = np.exp2(np.maximum(ex - 4.0, -9.0))          # 3 fraction bits; steps of 2^-9 below 2^-6
    return np.round(x / ulp) * ulp


def append(codes, scales, k, v, slots, fmt: str):
    """Write k, v [N, H, D] at `slots` (-1: skipped) into codes [NB, 2, H, block, D] (numbers, fp64)
    and scales [NB, 2, H], in place.  NaN is held as 0, an infinity as QMAX of the finite values' scale."""
    block = codes.shape[3]
    i, N = 0, len(slots)
    while i < N:
        if slots[i] < 0:
            i += 1
            continue
        page, off = divmod(int(slots[i]), block)
        j = i + 1
        while j < N and slots[j] == slots[i] + (j - i) and int(slots[j]) // block == page:
            j += 1
        for s, x in enumerate((k, v)):
            for h in range(codes.shape[2]):
                new = np.asarray(x[i:j, h], dtype=np.float64)
                new = np.where(np.isnan(new), 0.0, new)
                fin = np.abs(new[np.isfinite(new)])
                sc = 2.0 ** scale_exponent(float(fin.max()) if fin.size else 0.0, fmt)
                if off > 0:
                    old = float(scales[page, s, h])
                    sc = max(sc, old)
                    codes[page, s, h, :off] = quantise(codes[page, s, h, :off] * (old / sc), fmt)
                codes[page, s, h, off:off + j - i] = quantise(new / sc, fmt)
                scales[page, s, h] = sc
        i = j


def attention(q, k, v, seen, scale: float):
    """q [n, D], k, v [T, D], seen [n] (query i sees positions below seen[i]) -> [n, D] in fp64."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    out = np.zeros_like(q)
    for i in range(q.shape[0]):
        t = max(0, min(int(seen[i]), k.shape[0]))
        if t == 0:
            continue
        s = (k[:t] @ q[i]) * scale
        p = np.exp(s - s.max())
        out[i] = (p[:, None] * v[:t]).sum(0) / p.sum()
    return out


def frequencies(rot: int, base: float, scaling=None, factor=1.0, original=8192.0, low=1.0, high=4.0):
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            turns = original * f / (2 * math.pi)
            if turns <= low:
                f = f / factor
            elif turns < high:
                x = (turns - low) / (high - low)
                f = x * f + (1 - x) * f / factor
        out.append(f)
    return out


def rotate(x, pos, freq, layout: str, amp: float = 1.0):
    """x [n, heads, D] at positions pos [n] -> the same in fp64."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    half = len(freq)
    for i, f in enumerate(freq):
        a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        t = np.asarray(pos, dtype=np.float64) * f
        c, s = amp * np.cos(t)[:, None], amp * np.sin(t)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out
