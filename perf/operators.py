"""The attention operators of a decode step, as cases that can be timed and compared.

Four operators that stand next to the beam step and the paged cache:

  tables   block tables and slot maps of ragged prompts, built on the GPU from request lengths
  append   new K/V rows written into the 8-bit paged cache (one power-of-two scale per page and head)
  attend   attention of 1..32 new tokens per row over that cache, pages shared by a sentence's beams
  cross    attention of decoder rows to an encoder's states of another length

`run` computes an operator in plain torch operations, or, where `own` is set, through this
framework's entry points.  `exact` gives the operators' definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
QMAX = {"int8": 127.0, "e4m3": 448.0}
E_LO, E_HI = -60, 60           # the range of the scales' exponents


def listed():
    return [
        # a small service: 8 prompts of a few hundred tokens, 4 beams each
        {"name": "tables_8x4", "op": "tables", "batch": 8, "W": 4, "lo": 0, "hi": 200, "block": 16, "extra": 4},
        # a large batch of chat prompts, one row a request
        {"name": "tables_1024x1", "op": "tables", "batch": 1024, "W": 1, "lo": 1, "hi": 4095, "block": 16, "extra": 16},
        # one decode step of 256 rows at ragged positions (8 KV heads x 128 dims)
        {"name": "append_step_256_e4m3", "op": "append", "fmt": "e4m3", "src": "bf16", "batch": 256, "n_new": 1, "lo": 1,
         "hi": 1000, "H": 8, "D": 128, "block": 16},
        # the prompts of 64 sentences of about 1000 tokens
        {"name": "append_prompt_64_i8", "op": "append", "fmt": "int8", "src": "bf16", "batch": 64, "n_new": 0, "lo": 900,
         "hi": 1100, "H": 8, "D": 128, "block": 16},
        # small ragged prompts of a model with odd sizes, fp32 activations
        {"name": "append_prompt_7_odd", "op": "append", "fmt": "e4m3", "src": "f32", "batch": 7, "n_new": 0, "lo": 0,
         "hi": 333, "H": 5, "D": 48, "block": 24},
        # one sentence, 4 beams, a short context: the smallest call, where latency counts
        {"name": "attend_1x4_short", "op": "attend", "fmt": "int8", "batch": 1, "W": 4, "n_q": 1, "Hq": 8, "Hkv": 8, "D": 64,
         "lo": 100, "hi": 130, "gen": 20, "block": 16, "L": 2},
        # 64 sentences x 4 beams after prompts of about 1000 tokens (32 query heads, 8 KV heads x 128 dims)
        {"name": "attend_64x4_beams", "op": "attend", "fmt": "e4m3", "batch": 64, "W": 4, "n_q": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "lo": 950, "hi": 1050, "gen": 64, "block": 16, "L": 1},
        # a blockwise verify call: 8 proposed tokens a row
        {"name": "attend_64_verify8", "op": "attend", "fmt": "int8", "batch": 64, "W": 1, "n_q": 8, "Hq": 32, "Hkv": 8,
         "D": 128, "lo": 1, "hi": 4000, "gen": 0, "block": 32, "L": 1},
        # one row over a long document
        {"name": "attend_1_long", "op": "attend", "fmt": "e4m3", "batch": 1, "W": 1, "n_q": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "lo": 250001, "hi": 250001, "gen": 0, "block": 64, "L": 1},
        # translation decode step: 128 sentences x 4 beams, 8 heads x 64 dims, sources of up to 256 tokens
        {"name": "cross_step_128x4", "op": "cross", "batch": 128, "W": 4, "n_q": 1, "Hq": 8, "Hkv": 8, "D": 64, "lo": 1,
         "hi": 256},
        # scoring whole targets against long sources
        {"name": "cross_score_16x1024", "op": "cross", "batch": 16, "W": 1, "n_q": 1024, "Hq": 16, "Hkv": 16, "D": 64,
         "lo": 1000, "hi": 2048},
        # a prompt of a wide model with grouped heads against a few long sources
        {"name": "cross_prompt_4x500_gqa", "op": "cross", "batch": 4, "W": 1, "n_q": 500, "Hq": 32, "Hkv": 8, "D": 128,
         "lo": 500, "hi": 4000},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "cross", "cross"])
    if op == "tables":
        batch = _log_int(rng, 1, 1024)
        hi = _log_int(rng, 1, 4095)
        return {"op": op, "batch": batch, "W": rng.choice([1, 2, 4, 5]) if batch <= 256 else 1, "lo": rng.randint(0, hi), "hi": hi,
                "block": rng.choice([8, 16, 16, 32, 64]), "extra": rng.randint(1, 16)}
    if op == "append":
        step = rng.random() < 0.5
        return {"op": op, "fmt": rng.choice(["int8", "e4m3"]), "src": rng.choice(["bf16", "bf16", "f32"]),
                "batch": _log_int(rng, 1, 256 if step else 64), "n_new": _log_int(rng, 1, 32) if step else 0,
                "lo": rng.randint(0, 40), "hi": _log_int(rng, 40, 1000), "H": rng.choice([1, 2, 5, 8]),
                "D": rng.choice([16, 48, 64, 80, 128]), "block": rng.choice([8, 16, 16, 24, 32, 64])}
    if op == "attend":
        W = rng.choice([1, 1, 2, 4, 5, 8])
        Hkv = rng.choice([1, 2, 4, 8])
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 4, 2000)
        return {"op": op, "fmt": rng.choice(["int8", "e4m3"]), "batch": batch, "W": W,
                "n_q": 1 if W > 1 else rng.choice([1, 2, 4, 7, 8, 16]), "Hq": Hkv * rng.choice([1, 2, 4, 8 if Hkv <= 4 else 1]),
                "Hkv": Hkv, "D": rng.choice([32, 64, 80, 128, 128]), "lo": rng.randint(0, hi), "hi": hi,
                "gen": _log_int(rng, 1, 64) if W > 1 else 0, "block": rng.choice([8, 16, 16, 32, 64]), "L": rng.choice([1, 2])}
    long_q = rng.random() < 0.5
    Hkv = rng.choice([1, 4, 8])
    hi = _log_int(rng, 8, 2048)
    W = 1 if long_q else rng.choice([1, 2, 4, 5, 16])
    return {"op": op, "batch": _log_int(rng, 1, 8 if long_q else 128), "W": W,
            "n_q": _log_int(rng, 17, 700) if long_q else rng.choice([1, 1, 2, 8]) if W <= 2 else 1, "Hq": Hkv * rng.choice([1, 2]), "Hkv": Hkv,
            "D": rng.choice([32, 64, 64, 80, 128]), "lo": rng.randint(0, hi), "hi": hi}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _lengths(batch, lo, hi):
    """The request lengths before their order is drawn: evenly spread over [lo, hi]."""
    if batch == 1:
        return [hi]
    return [lo + (hi - lo) * i // (batch - 1) for i in range(batch)]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _mixed(case, seed):
    """The case's lengths in an order drawn from the seed (a host list)."""
    lens = _lengths(case["batch"], case["lo"], case["hi"])
    g = torch.Generator()
    g.manual_seed(seed)
    return [lens[i] for i in torch.randperm(len(lens), generator=g).tolist()]


def _exponent(amax, fmt):
    """The smallest integer e with amax <= QMAX 2^e, in [E_LO, E_HI]."""
    m, x = torch.frexp(amax)
    bits, top = (7, 0.9921875) if fmt == "int8" else (9, 0.875)      # QMAX = top 2^bits
    e = x.to(torch.int32) - bits + (m > top).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, E_LO)).clamp(E_LO, E_HI)


def _round(x, fmt):
    """x rounded to the format's nearest code (ties to even), as the codes' numbers."""
    x = x.clamp(-QMAX[fmt], QMAX[fmt])
    return torch.round(x) if fmt == "int8" else x.to(torch.float8_e4m3fn).float()


def _held(codes, fmt):
    """Code numbers as the cache's 8-bit elements."""
    return codes.to(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def _pow2(e):
    """2^e in fp32, from its bit pattern (exact)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantised_pages(n, H, block, D, fmt, g):
    """Pages of a cache in use: keys and values [n, 2, H, block, D] with their scales [n, 2, H]."""
    codes = torch.empty(n, 2, H, block, D, dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(n, 2, H, dtype=torch.float32, device=DEV)
    head = torch.exp(torch.randn(2, H, 1, 1, device=DEV, generator=g) * 0.5)
    step = max(1, (1 << 26) // (2 * H * block * D))
    for i in range(0, n, step):
        x = torch.randn(min(step, n - i), 2, H, block, D, device=DEV, generator=g) * head
        e = _exponent(x.abs().amax(dim=(3, 4)), fmt)
        scales[i:i + step] = _pow2(e)
        codes[i:i + step] = _held(_round(x * _pow2(-e[..., None, None]), fmt), fmt)
    return codes, scales


def _beam_pages(case, lens, seed):
    """Which page each row's tables name after `gen` generated positions: the beams of a sentence
    share its prompt's full pages, diverge in the page they write and follow their parents when
    they are reordered (every 8 positions).  Returns (ids [R][pages], parents {t: [R]}, n)."""
    W, block, gen = case["W"], case["block"], case["gen"]
    g = torch.Generator()
    g.manual_seed(seed + 1)
    R = case["batch"] * W
    parents = {}
    for t in range(8, gen, 8):
        draw_ = torch.randint(0, W, (case["batch"], W), generator=g).sort(dim=1).values
        parents[t] = (draw_ + torch.arange(case["batch"])[:, None] * W).reshape(R).tolist()
    ids, n = [], 0
    for b, P in enumerate(lens):
        pages = -(-P // block)
        rows = [list(range(n, n + pages)) for _ in range(W)]
        n += pages
        for t in range(gen):
            if t in parents:
                rows = [list(rows[parents[t][b * W + w] - b * W]) for w in range(W)]
            i = (P + t) // block
            seen = set()
            for w in range(W):                          # the page being written is each row's own
                if len(rows[w]) == i:
                    rows[w].append(n)
                    n += 1
                elif rows[w][i] in seen:
                    rows[w][i] = n
                    n += 1
                seen.add(rows[w][i])
        ids += rows
    return ids, parents, n


def prepare(case, seed):
    return {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend,
            "cross": _prepare_cross}[case["op"]](case, seed)


def _tables_geometry(case):
    pages = -(-case["hi"] // case["block"])
    return pages + case["W"] * case["extra"], pages + case["extra"]      # pages a sentence owns, table entries a row


def _prepare_tables(case, seed):
    lens = _mixed(case, seed)
    S, MB = _tables_geometry(case)
    st = {"case": case, "S": S, "MB": MB, "total": sum(lens), "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if own:
        import verify_bs_step_gb300 as vbs
        st["kv"] = vbs.PagedKV(case["batch"], case["W"], 1, 1, 16, blocks_per_sentence=S, max_blocks=MB,
                               block=case["block"], dtype=torch.bfloat16)
    return st


def _prepare_append(case, seed):
    """Prompts written whole (n_new = 0), or n_new tokens after each row's context.  Request b owns
    the pages [b S, (b+1) S) and its j-th page is b S + j."""
    lens = _mixed(case, seed)
    g = _gen(seed)
    H, D, block, n_new = case["H"], case["D"], case["block"], case["n_new"]
    counts = [n_new] * len(lens) if n_new else lens
    starts = lens if n_new else [0] * len(lens)
    S = max(1, -(-(case["hi"] + n_new) // block))
    NB, N = len(lens) * S, sum(counts)
    first = torch.tensor(starts, device=DEV)
    cnt = torch.tensor(counts, device=DEV)
    req = torch.repeat_interleave(torch.arange(len(lens), device=DEV), cnt, output_size=N)
    at = torch.arange(N, device=DEV) - (torch.cumsum(cnt, 0) - cnt)[req] + first[req]
    slots = (req * S + at // block) * block + at % block
    # what is read back: every position of the pages that were written to, up to the last one
    low = first // block * block
    back = first + cnt - low
    M = int(back.sum())
    rq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), back, output_size=M)
    ra = torch.arange(M, device=DEV) - (torch.cumsum(back, 0) - back)[rq] + low[rq]
    src = torch.bfloat16 if case["src"] == "bf16" else torch.float32
    head = torch.exp(torch.randn(2, 1, H, 1, device=DEV, generator=g) * 0.5)
    tok = torch.exp(torch.randn(N, 1, 1, device=DEV, generator=g) * 0.7)
    # one projection's output: K and V are slices of it, as a model has them
    kv_new = torch.empty(N, 2, H, D, dtype=src, device=DEV)
    for i in (0, 1):
        kv_new[:, i] = (torch.randn(N, H, D, device=DEV, generator=g) * head[i] * tok).to(src)
    codes, scales = _quantised_pages(NB, H, block, D, case["fmt"], g) if n_new else (
        torch.zeros(NB, 2, H, block, D, dtype=torch.int8 if case["fmt"] == "int8" else torch.float8_e4m3fn, device=DEV),
        torch.zeros(NB, 2, H, dtype=torch.float32, device=DEV))
    st = {"case": case, "k": kv_new[:, 0], "v": kv_new[:, 1], "slots": slots, "S": S,
          "back": (rq * S + ra // block) * block + ra % block}
    if own:
        import verify_bs_step_gb300 as vbs
        kv = vbs.PagedKV8(len(lens), 1, 1, H, D, heads=H, blocks_per_sentence=S, max_blocks=S, block=block,
                          dtype=codes.dtype, pool=codes.view(NB, 1, 2, H, block, D), scales=scales.view(NB, 1, 2, H))
        st["kv"] = kv
    else:
        st["codes"], st["scales"] = codes, scales
    return st


def _prepare_attend(case, seed):
    lens = _mixed(case, seed)
    g = _gen(seed)
    W, H, D, block, gen, n_q = case["W"], case["Hkv"], case["D"], case["block"], case["gen"], case["n_q"]
    ids, parents, n = _beam_pages(case, lens, seed)
    codes, scales = _quantised_pages(max(n, 1), H, block, D, case["fmt"], g)
    R = len(lens) * W
    ctx = torch.tensor([p + gen for p in lens for _ in range(W)], dtype=torch.int32, device=DEV)
    q = torch.randn(R, n_q, case["Hq"], D, device=DEV, generator=g).mul_(1.5).to(torch.bfloat16)
    most = max([len(r) for r in ids] + [1])
    st = {"case": case, "q": q, "ctx": ctx}
    rows = torch.tensor([r + [-1] * (most - len(r)) for r in ids], device=DEV)
    if own:
        import verify_bs_step_gb300 as vbs
        MB = most + 1
        S = max(-(-p // block) for p in lens) + W * (gen // block + 3)
        pool = torch.zeros(len(lens) * S, case["L"], 2, H, block, D, dtype=codes.dtype, device=DEV)
        kv = vbs.PagedKV8(len(lens), W, case["L"], H, D, heads=case["Hq"], max_q=n_q, blocks_per_sentence=S,
                          max_blocks=MB, block=block, dtype=codes.dtype, pool=pool)
        kv.build(torch.tensor(lens, dtype=torch.int32, device=DEV))
        for t in range(gen):
            if t in parents:
                kv.reorder(torch.tensor(parents[t], dtype=torch.int32, device=DEV), t)
            else:
                kv.prepare(t)
        have = rows >= 0
        at = kv.table()[:, :most].long()[have]
        kv.pool[:, -1].view(torch.uint8)[at] = codes.view(torch.uint8)[rows[have]]
        kv.scales[:, -1][at] = scales[rows[have]]
        st["kv"] = kv
    else:
        st["codes"], st["scales"], st["rows"] = codes, scales, rows
    return st


def _prepare_cross(case, seed):
    lens = _mixed(case, seed)
    g = _gen(seed)
    B, W, n_q, Hq, H, D, S = case["batch"], case["W"], case["n_q"], case["Hq"], case["Hkv"], case["D"], max(1, case["hi"])
    # the encoder's K and V: two slices of one projection of its states, [B, S, 2, H, D]
    kv = torch.randn(B, S, 2, H, D, device=DEV, generator=g, dtype=torch.float32).to(torch.bfloat16)
    st = {"case": case, "q": torch.randn(B * W, n_q, Hq, D, device=DEV, generator=g).mul_(1.5).to(torch.bfloat16),
          "k": kv[:, :, 0], "v": kv[:, :, 1], "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if own:
        import verify_bs_step_gb300 as vbs
        st["op"] = vbs.CrossAttention(B, W, Hq, D, kv_heads=H, max_q=n_q, max_len=S)
    return st


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(state):
    return (_RUN_OWN if own else _RUN)[state["case"]["op"]](state)


def _own_tables(st):
    kv = st["kv"]
    slots, pos, row, cu = kv.build(st["lens"], st["total"])
    return list(kv.views()) + [slots, pos, row, cu]


def _own_append(st):
    kv = st["kv"]
    kv.append(0, st["k"], st["v"], st["slots"])
    k, v = kv.read(0, st["back"])
    return [k, v, kv.scales[:, 0]]


def _own_attend(st):
    kv = st["kv"]
    kv.plan(st["ctx"], st["q"].shape[1])
    return kv.attend(st["case"]["L"] - 1, st["q"])


def _own_cross(st):
    return st["op"].attend(st["q"], st["k"], st["v"], st["lens"])


def _plain_tables(st):
    c, S, MB, lens = st["case"], st["S"], st["MB"], st["lens"]
    B, W, block = c["batch"], c["W"], c["block"]
    i32 = torch.int32
    pages = (lens + block - 1) // block
    b = torch.arange(B, device=DEV)
    j = torch.arange(MB, device=DEV)
    table = torch.where(j < pages[:, None], b[:, None] * S + j, -1).to(i32).repeat_interleave(W, 0)
    nblk = pages.to(i32).repeat_interleave(W)
    s = torch.arange(S, device=DEV)
    refcnt = torch.where(s < pages[:, None], W, 0).to(i32).reshape(-1)
    stack = (b[:, None] * S + S - 1 - s).to(i32).reshape(-1)
    top = (S - pages).to(i32)
    cu = torch.zeros(B + 1, dtype=i32, device=DEV)
    cu[1:] = torch.cumsum(lens, 0)
    req = torch.repeat_interleave(b, lens, output_size=st["total"])
    pos = torch.arange(st["total"], device=DEV) - cu[req]
    slots = table[req * W, pos // block].long() * block + pos % block
    return [table, nblk, refcnt, stack, top, slots, pos.to(i32), (req * W).to(i32), cu]


def _plain_append(st):
    c = st["case"]
    fmt, block, H, D = c["fmt"], c["block"], c["H"], c["D"]
    codes, scales, slots = st["codes"], st["scales"], st["slots"]
    NB = scales.shape[0]
    x = torch.stack((st["k"], st["v"]), 1).float()                   # [N, 2, H, D]
    page, off = slots // block, slots % block
    first = torch.full((NB,), block, device=DEV).scatter_reduce(0, page, off, "amin")
    hit = torch.unique(page)
    rows = x.abs().amax(-1).reshape(-1, 2 * H)
    amax = torch.zeros(NB, 2 * H, device=DEV).scatter_reduce(0, page[:, None].expand_as(rows), rows, "amax")[hit]
    e = _exponent(amax.view(-1, 2, H), fmt)
    old = scales[hit]
    e_old = torch.frexp(old).exponent.to(torch.int32) - 1
    keep = (first[hit] > 0)[:, None, None]
    e = torch.where(keep, torch.maximum(e, e_old), e)
    was = codes.view(torch.uint8)[hit].view(codes.dtype).float()
    shifted = _held(_round(was * torch.where(keep, old / _pow2(e), 1.0)[..., None, None], fmt), fmt)
    earlier = torch.arange(block, device=DEV) < first[hit][:, None]
    raw = codes.view(torch.uint8)
    raw[hit] = torch.where(earlier[:, None, None, :, None], shifted.view(torch.uint8), raw[hit])
    scales[hit] = _pow2(e)
    new = _held(_round(x / scales[page][..., None], fmt), fmt)       # a power of two: exact
    raw[page, :, :, off] = new.view(torch.uint8)
    bp, bo = st["back"] // block, st["back"] % block
    vals = raw[bp, :, :, bo].view(codes.dtype).float() * scales[bp][..., None]
    return [vals[:, 0].to(torch.bfloat16), vals[:, 1].to(torch.bfloat16), scales]


def _plain_attend(st):
    c, q, ctx, rows = st["case"], st["q"].float(), st["ctx"], st["rows"]
    R, n_q, Hq, D = q.shape
    H, G, block = c["Hkv"], Hq // c["Hkv"], c["block"]
    at = rows.clamp(min=0)
    kv = st["codes"].view(torch.uint8)[at].view(st["codes"].dtype).float() * st["scales"][at][..., None, None]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, R, H, -1, D)        # [2, R, H, positions, D]
    q = q.view(R, n_q, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, n_q * G, D)
    s = torch.matmul(q, kv[0].transpose(-1, -2)) / math.sqrt(D)
    limit = ctx[:, None] - n_q + 1 + torch.arange(n_q, device=DEV)   # [R, n_q]
    dead = (torch.arange(s.shape[-1], device=DEV) >= limit[..., None]).repeat_interleave(G, 1)[:, None]
    s = s.masked_fill(dead, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[1]) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(R, H, n_q, G, D).permute(0, 2, 1, 3, 4).reshape(R, n_q, Hq, D).to(torch.bfloat16)


def _plain_cross(st):
    c, q, k, v, lens = st["case"], st["q"].float(), st["k"].float(), st["v"].float(), st["lens"]
    B, W, n_q, Hq, H, D = c["batch"], c["W"], c["n_q"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // H
    q = q.view(B, W * n_q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, W * n_q * G, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(D)
    dead = (torch.arange(s.shape[-1], device=DEV) >= lens[:, None])[:, None, None]
    s.masked_fill_(dead, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, H, W * n_q, G, D).permute(0, 2, 1, 3, 4).reshape(B * W, n_q, Hq, D).to(torch.bfloat16)


_RUN = {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend, "cross": _plain_cross}
_RUN_OWN = {"tables": _own_tables, "append": _own_append, "attend": _own_attend, "cross": _own_cross}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------

def work(case):
    op, lens = case["op"], _lengths(case["batch"], case["lo"], case["hi"])
    B, total = len(lens), sum(lens)
    if op == "tables":
        S, MB = _tables_geometry(case)
        R = B * case["W"]
        # lengths; the tables, counts and free stacks; slot, position and row of every token
        return {"bytes": 4 * B + 4 * R * (MB + 1) + 8 * B * S + 16 * total + 4 * (B + 1), "flops": 0}
    if op == "append":
        H, D, n_new, block = case["H"], case["D"], case["n_new"], case["block"]
        n = B * n_new if n_new else total
        back = sum(p % block + n_new for p in lens) if n_new else total
        pages = sum((p + n_new - 1) // block - p // block + 1 for p in lens) if n_new else sum(-(-p // block) for p in lens)
        src = 2 if case["src"] == "bf16" else 4
        # rows in, codes out; codes read back, values out; slots and scales
        return {"bytes": 2 * H * D * (n * (src + 1) + back * 3) + 8 * (n + back) + 8 * H * pages, "flops": 4 * H * D * n}
    if op == "attend":
        W, H, Hq, D, n_q, gen, block = case["W"], case["Hkv"], case["Hq"], case["D"], case["n_q"], case["gen"], case["block"]
        # every distinct cached position once: a page that several beams of a sentence share counts once
        ids = _beam_pages(case, lens, 0)[0]
        cached = 0
        for b, p in enumerate(lens):
            named = {(i, j) for r in ids[b * W:(b + 1) * W] for j, i in enumerate(r)}
            cached += sum(max(0, min(block, p + gen - j * block)) for _, j in named)
        pairs = sum(max(0, p + gen - i) for p in lens for i in range(n_q)) * W * Hq
        return {"bytes": 2 * H * (D * cached + 4 * (cached // block + 1)) + 4 * B * W * n_q * Hq * D, "flops": 4 * D * pairs}
    W, H, Hq, D, n_q = case["W"], case["Hkv"], case["Hq"], case["D"], case["n_q"]
    return {"bytes": 4 * H * D * total + 4 * B * W * n_q * Hq * D, "flops": 4 * D * total * W * n_q * Hq}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------

def _plain_state(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _softmax_rows64(q, k, v, scale, valid):
    """softmax(scale q k^T) v over the positions below valid[i] of each query i, in 64 bits; zeros where there are none."""
    s = (q @ k.T) * scale
    keep = torch.arange(k.shape[0], device=q.device)[None, :] < valid[:, None]
    s = torch.where(keep, s, -math.inf)
    top = s.max(dim=1, keepdim=True).values.clamp(min=-1e300)
    p = torch.where(keep, torch.exp(s - top), 0.0)
    z = p.sum(dim=1, keepdim=True)
    return torch.where(z > 0, (p @ v) / z.clamp(min=1e-300), 0.0)


def _exact_append(case, seed):
    st = _plain_state(case, seed)
    block, fmt, H = case["block"], case["fmt"], case["H"]
    top = QMAX[fmt]
    pool = st["codes"].view(torch.uint8).clone()
    dt = st["codes"].dtype
    scales = st["scales"].double()
    slots = st["slots"].cpu()
    x = torch.stack((st["k"], st["v"]), 1).double()
    # the runs of tokens that fall into one page, one after the other
    page = slots // block
    starts = [0] + [i for i in range(1, len(page)) if page[i] != page[i - 1]] if len(page) else []
    if len(starts) > 6000:
        return None
    for i, a in enumerate(starts):
        z = starts[i + 1] if i + 1 < len(starts) else len(page)
        p, o = int(page[a]), int(slots[a] % block)
        rows = x[a:z].permute(1, 2, 0, 3)                              # [2, H, n, D]
        need = rows.abs().amax(dim=(2, 3)).tolist()
        was = scales[p].tolist()
        now = [[_scale64(need[kv][h], top, was[kv][h] if o else 0.0) for h in range(H)] for kv in (0, 1)]
        s = torch.tensor(now, dtype=torch.float64, device=DEV)
        if o:
            held = pool[p, :, :, :o].view(dt).double() * (scales[p] / s)[..., None, None]
            pool[p, :, :, :o] = _code64(held, fmt).view(torch.uint8)
        pool[p, :, :, o:o + z - a] = _code64(rows / s[..., None, None], fmt).view(torch.uint8)
        scales[p] = s
    bp, bo = st["back"] // block, st["back"] % block
    vals = pool[bp, :, :, bo].view(dt).double() * scales[bp][..., None]
    return [vals[:, 0], vals[:, 1], scales]


def _scale64(amax, top, was):
    """The smallest power of two s, not below `was`, with amax <= top s."""
    e = E_LO
    if amax > 0:
        e = math.ceil(math.log2(amax / top))
        while amax > top * 2.0 ** e:
            e += 1
        while amax <= top * 2.0 ** (e - 1):
            e -= 1
    return max(2.0 ** max(E_LO, min(E_HI, e)), was)


def _code64(x, fmt):
    """The nearest code of 64-bit values, ties to even."""
    if fmt == "int8":
        return torch.round(x.clamp(-127, 127)).to(torch.int8)
    # e4m3: 3 fraction bits above 2^-6, steps of 2^-9 below
    _, ex = torch.frexp(x)
    ulp = (((ex - 4).clamp(min=-9).long() + 1023) << 52).view(torch.float64)
    return (torch.round(x / ulp) * ulp).clamp(-448, 448).float().to(torch.float8_e4m3fn)


def _exact_attend(case, seed):
    st = _plain_state(case, seed)
    q, ctx, rows = st["q"].double(), st["ctx"].tolist(), st["rows"].tolist()
    H, n_q, Hq, D = case["Hkv"], case["n_q"], case["Hq"], case["D"]
    G = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    step = torch.arange(n_q, device=DEV).repeat_interleave(G)
    if q.shape[0] * H > 4096:
        return None
    for r in range(q.shape[0]):
        ids = [i for i in rows[r] if i >= 0]
        if not ids:
            continue
        at = torch.tensor(ids, device=DEV)
        codes = st["codes"].view(torch.uint8)[at].view(st["codes"].dtype).double()      # [pages, 2, H, block, D]
        vals = codes * st["scales"][at].double()[..., None, None]
        for h in range(H):
            k = vals[:, 0, h].reshape(-1, D)
            v = vals[:, 1, h].reshape(-1, D)
            mine = q[r, :, h * G:(h + 1) * G].reshape(n_q * G, D)
            o = _softmax_rows64(mine, k, v, D ** -0.5, ctx[r] - n_q + 1 + step)
            out[r, :, h * G:(h + 1) * G] = o.view(n_q, G, D)
    return out


def _exact_cross(case, seed):
    st = _plain_state(case, seed)
    B, W, n_q, Hq, H, D = case["batch"], case["W"], case["n_q"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // H
    q = st["q"].view(B, W * n_q, Hq, D)
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lens = st["lens"].tolist()
    for b in range(B):
        for h in range(H):
            k, v = st["k"][b, :lens[b], h].double(), st["v"][b, :lens[b], h].double()
            if not lens[b]:
                continue
            for i in range(G):
                mine = q[b, :, h * G + i].double()
                out[b, :, h * G + i] = _softmax_rows64(mine, k, v, D ** -0.5,
                                                       torch.full((W * n_q,), lens[b], device=DEV))
    return out.view(B * W, n_q, Hq, D)


def exact(case, seed):
    if case["op"] == "tables":
        return None                                # whole numbers only
    return {"append": _exact_append, "attend": _exact_attend, "cross": _exact_cross}[case["op"]](case, seed)
