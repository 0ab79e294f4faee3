"""The operators around a 16-bit paged cache, as cases that can be timed and compared.

Three operators of a decoder whose keys and values are held in bf16:

  rotary   rotary positions of queries and keys, with the new K/V rows written into the paged cache in the same
           call (prompts and steps), or applied alone
  prompt   attention of whole packed prompts to themselves, causal or (an encoder's) in both directions, with
           grouped heads
  paged    attention of 1..32 new tokens per row over the paged cache, pages shared by a sentence's beams

`run` computes an operator in plain torch operations, or, where `own` is set, through this framework's entry
points.  `exact` gives the operators' definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


def listed():
    return [
        # one sentence's 4 beams take a step: the smallest call, where latency counts
        {"name": "rotary_step_4", "op": "rotary", "mode": "step", "src": "bf16", "batch": 4, "lo": 100, "hi": 130, "Hq": 8, "H": 8,
         "D": 64, "rot": 64, "layout": "half", "scaling": "none", "block": 16},
        # a step of 64 sentences x 4 beams (32 query heads, 8 KV heads x 128 dims), contexts scaled to 8 times their length
        {"name": "rotary_step_256", "op": "rotary", "mode": "step", "src": "bf16", "batch": 256, "lo": 1, "hi": 60000, "Hq": 32,
         "H": 8, "D": 128, "rot": 128, "layout": "half", "scaling": "parts", "block": 16},
        # the prompts of 64 sentences of about 1000 tokens
        {"name": "rotary_prompt_64", "op": "rotary", "mode": "prompt", "src": "bf16", "batch": 64, "lo": 900, "hi": 1100, "Hq": 32,
         "H": 8, "D": 128, "rot": 128, "layout": "half", "scaling": "none", "block": 16},
        # fp32 activations of odd sizes, pairs side by side, part of the head, far into a document, no cache
        {"name": "rotary_apply_odd", "op": "rotary", "mode": "apply", "src": "f32", "batch": 3, "lo": 700000, "hi": 701234,
         "Hq": 9, "H": 3, "D": 80, "rot": 36, "layout": "interleaved", "scaling": "linear", "block": 16},
        # a few short prompts of a small model
        {"name": "prompt_8_short", "op": "prompt", "batch": 8, "lo": 0, "hi": 60, "Hq": 8, "H": 8, "D": 64, "causal": True},
        # an encoder's own attention over 128 ragged sentences
        {"name": "prompt_128_encoder", "op": "prompt", "batch": 128, "lo": 1, "hi": 256, "Hq": 8, "H": 8, "D": 64,
         "causal": False},
        # the prompts of 64 sentences of about 1000 tokens (32 query heads, 8 KV heads x 128 dims)
        {"name": "prompt_64x1000", "op": "prompt", "batch": 64, "lo": 900, "hi": 1100, "Hq": 32, "H": 8, "D": 128, "causal": True},
        # one long document
        {"name": "prompt_1_long", "op": "prompt", "batch": 1, "lo": 16001, "hi": 16001, "Hq": 32, "H": 8, "D": 128,
         "causal": True},
        # one sentence, 4 beams, a short context
        {"name": "paged_1x4_short", "op": "paged", "batch": 1, "W": 4, "n_q": 1, "Hq": 8, "H": 8, "D": 64, "lo": 100, "hi": 130,
         "gen": 20, "block": 16, "L": 2},
        # 64 sentences x 4 beams after prompts of about 1000 tokens
        {"name": "paged_64x4_beams", "op": "paged", "batch": 64, "W": 4, "n_q": 1, "Hq": 32, "H": 8, "D": 128, "lo": 950,
         "hi": 1050, "gen": 64, "block": 16, "L": 1},
        # a blockwise verify call: 8 proposed tokens a row
        {"name": "paged_64_verify8", "op": "paged", "batch": 64, "W": 1, "n_q": 8, "Hq": 32, "H": 8, "D": 128, "lo": 1, "hi": 2500,
         "gen": 0, "block": 32, "L": 1},
        # one row over a long document
        {"name": "paged_1_long", "op": "paged", "batch": 1, "W": 1, "n_q": 1, "Hq": 32, "H": 8, "D": 128, "lo": 100003,
         "hi": 100003, "gen": 0, "block": 64, "L": 1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "prompt", "prompt", "paged", "paged"])
    if op == "rotary":
        mode = rng.choice(["step", "prompt", "apply"])
        D = rng.choice([32, 64, 80, 128, 128])
        H = rng.choice([1, 2, 5, 8])
        lo = rng.randint(0, 60000 if mode == "step" else 40)
        return {"op": op, "mode": mode, "src": rng.choice(["bf16", "bf16", "f32"]),
                "batch": _log_int(rng, 1, 256 if mode == "step" else 48), "lo": lo, "hi": lo + _log_int(rng, 1, 1000), "Hq": H * rng.choice([1, 2, 4]),
                "H": H, "D": D, "rot": rng.choice([D, D, D // 2, D - 6]), "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "parts"]), "block": rng.choice([8, 16, 16, 24, 32, 64])}
    if op == "prompt":
        batch = _log_int(rng, 1, 128)
        H = rng.choice([1, 2, 4, 8])
        hi = _log_int(rng, 1, int((6e7 / batch) ** 0.5))
        return {"op": op, "batch": batch, "lo": rng.randint(0, hi), "hi": hi, "Hq": H * rng.choice([1, 2, 3, 4, 8 if H <= 4 else 4]),
                "H": H, "D": rng.choice([32, 64, 64, 80, 128, 128]), "causal": rng.random() < 0.75}
    W = rng.choice([1, 1, 2, 4, 5, 8])
    H = rng.choice([1, 2, 4, 8])
    batch = _log_int(rng, 1, 64)
    hi = _log_int(rng, 4, min(1500, 250000 // (batch * W)))
    return {"op": op, "batch": batch, "W": W, "n_q": 1 if W > 1 else rng.choice([1, 2, 4, 7, 8, 16]),
            "Hq": H * rng.choice([1, 2, 4, 8 if H <= 4 else 1]), "H": H, "D": rng.choice([32, 64, 80, 128, 128]),
            "lo": rng.randint(0, hi), "hi": hi, "gen": _log_int(rng, 1, 64) if W > 1 else 0, "block": rng.choice([8, 16, 16, 32, 64]),
            "L": rng.choice([1, 2])}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _lengths(case):
    """The requests' lengths before their order is drawn: evenly spread over [lo, hi]."""
    batch, lo, hi = case["batch"], case["lo"], case["hi"]
    if batch == 1:
        return [hi]
    return [lo + (hi - lo) * i // (batch - 1) for i in range(batch)]


def _mixed(case, seed):
    """The case's lengths in an order drawn from the seed (a host list)."""
    lens = _lengths(case)
    g = torch.Generator()
    g.manual_seed(seed)
    return [lens[i] for i in torch.randperm(len(lens), generator=g).tolist()]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    return {"rotary": _prepare_rotary, "prompt": _prepare_prompt, "paged": _prepare_paged}[case["op"]](case, seed)


# the parameters of the scaled frequencies, by the case's "scaling"
_SCALING = {"none": {}, "linear": {"scaling": "linear", "factor": 4.0}, "base": {"scaling": "base", "factor": 4.0},
            "parts": {"scaling": "parts", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0, "amplitude": 1.2}}
_BASE = {"none": 10000.0, "linear": 10000.0, "base": 10000.0, "parts": 500000.0}


def _spans(case, lens):
    """Per request: the first position and the number of tokens (a step: one token at `len`; else: a span that
    starts at lo, of the lengths' differences where positions are far, or whole prompts)."""
    if case["mode"] == "step":
        return lens, [1] * len(lens)
    if case["mode"] == "apply":
        return [case["lo"]] * len(lens), [n - case["lo"] for n in lens]
    return [0] * len(lens), lens


def _prepare_rotary(case, seed):
    """Request b owns the pages [b S, (b+1) S) of the cache; position p goes to its page p // block, around S."""
    lens = _mixed(case, seed)
    g = _gen(seed)
    H, Hq, D, block = case["H"], case["Hq"], case["D"], case["block"]
    starts, counts = _spans(case, lens)
    N = sum(counts)
    cnt = torch.tensor(counts, device=DEV)
    req = torch.repeat_interleave(torch.arange(len(lens), device=DEV), cnt, output_size=N)
    pos = torch.arange(N, device=DEV) - (torch.cumsum(cnt, 0) - cnt)[req] + torch.tensor(starts, device=DEV)[req]
    src = BF16 if case["src"] == "bf16" else torch.float32
    # one projection's output: queries, keys and values are slices of it, as a model has them
    qkv = torch.randn(N, Hq + 2 * H, D, device=DEV, generator=g).to(src)
    st = {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + H], "v": qkv[:, Hq + H:], "pos": pos.to(torch.int32)}
    if case["mode"] != "apply":
        S = 2 if case["mode"] == "step" else max(1, -(-case["hi"] // block))
        st["slots"] = (req * S + pos // block % S) * block + pos % block
        st["pool"] = torch.randn(len(lens) * S, 1, 2, H, block, D, device=DEV, generator=g).to(BF16)
    if own:
        import verify_bs_step_gb300 as vbs
        st["rope"] = vbs.Rotary(D, rot=case["rot"], base=_BASE[case["scaling"]], layout=case["layout"], **_SCALING[case["scaling"]])
        if case["mode"] != "apply":
            st["kv"] = vbs.PagedKV16(len(lens), 1, 1, H, D, heads=Hq, blocks_per_sentence=S, max_blocks=S, block=block, pool=st["pool"])
    return st


def _prepare_prompt(case, seed):
    lens = _mixed(case, seed)
    g = _gen(seed)
    H, Hq, D = case["H"], case["Hq"], case["D"]
    N = sum(lens)
    qkv = torch.randn(N, Hq + 2 * H, D, device=DEV, generator=g)
    qkv[:, :Hq] *= 1.5
    qkv = qkv.to(BF16)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st = {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + H], "v": qkv[:, Hq + H:], "lens": lens, "starts": cu[:-1],
          "cu": torch.tensor(cu, dtype=torch.int32, device=DEV)}
    if own:
        import verify_bs_step_gb300 as vbs
        st["op"] = vbs.PromptAttention(Hq, D, kv_heads=H)
    else:
        # requests whose padded scores fit together: (first token, lengths) as tensors, the longest of them
        st["groups"], at = [], 0
        while at < len(lens):
            to, top = at, 0
            while to < len(lens) and (to == at or (to + 1 - at) * Hq * max(top, lens[to]) ** 2 <= 1 << 27):
                top = max(top, lens[to])
                to += 1
            st["groups"].append((torch.tensor(cu[at:to], device=DEV), torch.tensor(lens[at:to], device=DEV), top))
            at = to
    return st


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
        chosen = torch.randint(0, W, (case["batch"], W), generator=g).sort(dim=1).values
        parents[t] = (chosen + torch.arange(case["batch"])[:, None] * W).reshape(R).tolist()
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


def _prepare_paged(case, seed):
    lens = _mixed(case, seed)
    g = _gen(seed)
    W, H, D, block, gen, n_q = case["W"], case["H"], case["D"], case["block"], case["gen"], case["n_q"]
    ids, parents, n = _beam_pages(case, lens, seed)
    pages = torch.randn(max(n, 1), 2, H, block, D, device=DEV, generator=g, dtype=torch.float32).to(BF16)
    R = len(lens) * W
    ctx = torch.tensor([p + gen for p in lens for _ in range(W)], dtype=torch.int32, device=DEV)
    q = torch.randn(R, n_q, case["Hq"], D, device=DEV, generator=g).mul_(1.5).to(BF16)
    most = max([len(r) for r in ids] + [1])
    st = {"case": case, "q": q, "ctx": ctx}
    rows = torch.tensor([r + [-1] * (most - len(r)) for r in ids], device=DEV)
    if own:
        import verify_bs_step_gb300 as vbs
        S = max(-(-p // block) for p in lens) + W * (gen // block + 3)
        pool = torch.zeros(len(lens) * S, case["L"], 2, H, block, D, dtype=BF16, device=DEV)
        kv = vbs.PagedKV16(len(lens), W, case["L"], H, D, heads=case["Hq"], max_q=n_q, blocks_per_sentence=S, max_blocks=most + 1,
                           block=block, pool=pool)
        kv.build(torch.tensor(lens, dtype=torch.int32, device=DEV))
        for t in range(gen):
            if t in parents:
                kv.reorder(torch.tensor(parents[t], dtype=torch.int32, device=DEV), t)
            else:
                kv.prepare(t)
        have = rows >= 0
        at = kv.table()[:, :most].long()[have]
        kv.pool[at, -1] = pages[rows[have]]
        st["kv"] = kv
    else:
        st["pages"], st["rows"] = pages, rows
    return st


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(state):
    return (_RUN_OWN if own else _RUN)[state["case"]["op"]](state)


def _own_rotary(st):
    mode = st["case"]["mode"]
    if mode == "apply":
        return list(st["rope"].apply(st["pos"], st["q"], st["k"]))
    if mode == "step":                                 # the step's keys are read from the cache alone
        q, _ = st["kv"].append(0, st["k"], st["v"], st["slots"], rotary=st["rope"], pos=st["pos"], q=st["q"])
        return [q, st["pool"]]
    k = torch.empty(st["k"].shape, dtype=st["k"].dtype, device=DEV)
    q, k = st["kv"].append(0, st["k"], st["v"], st["slots"], rotary=st["rope"], pos=st["pos"], q=st["q"], k_out=k)
    return [q, k, st["pool"]]


def _own_prompt(st):
    return st["op"].attend(st["q"], st["k"], st["v"], st["cu"], causal=st["case"]["causal"])


def _own_paged(st):
    kv = st["kv"]
    kv.plan(st["ctx"], st["q"].shape[1])
    return kv.attend(st["case"]["L"] - 1, st["q"])


def _frequencies(case):
    """Radians a position for each pair of rotated dims, and the factor on the rotated values."""
    rot, sc = case["rot"], case["scaling"]
    p = _SCALING[sc]
    base = _BASE[sc] * (p["factor"] ** (rot / (rot - 2)) if sc == "base" else 1.0)
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=DEV)
    if sc == "linear":
        f = f / p["factor"]
    if sc == "parts":
        # by the turns that a pair makes over the original length: few are stretched, many are left
        keep = ((p["original"] * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / p["factor"])
    return f, p.get("amplitude", 1.0)


def _plain_rotary(st):
    c = st["case"]
    rot = c["rot"]
    f, amp = _frequencies(c)
    angle = st["pos"].double()[:, None] * f                           # far positions: 64 bits
    cos, sin = (torch.cos(angle) * amp).float()[:, None], (torch.sin(angle) * amp).float()[:, None]

    def turned(x):
        y = x.float()
        out = y.clone()
        if c["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            out[..., :rot // 2] = a * cos - b * sin
            out[..., rot // 2:rot] = b * cos + a * sin
        else:
            a, b = y[..., :rot:2], y[..., 1:rot:2]
            out[..., :rot:2] = a * cos - b * sin
            out[..., 1:rot:2] = b * cos + a * sin
        return out

    q, k = turned(st["q"]), turned(st["k"])
    dt = st["q"].dtype
    if c["mode"] == "apply":
        return [q.to(dt), k.to(dt)]
    page, off = st["slots"] // c["block"], st["slots"] % c["block"]
    st["pool"][page, 0, 0, :, off] = k.to(BF16)
    st["pool"][page, 0, 1, :, off] = st["v"].to(BF16)
    return [q.to(dt), st["pool"]] if c["mode"] == "step" else [q.to(dt), k.to(dt), st["pool"]]


def _plain_softmax(s, dead):
    """Weights of scores, 0 where dead, and in rows that are dead throughout."""
    s = s.masked_fill(dead, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_prompt(st):
    c = st["case"]
    H, Hq, D = c["H"], c["Hq"], c["D"]
    G = Hq // H
    out = torch.zeros(st["q"].shape, dtype=BF16, device=DEV)
    for first, n, top in st["groups"]:
        if top == 0:
            continue
        B = len(n)
        j = torch.arange(top, device=DEV)
        there = j < n[:, None]                                        # [B, top]
        at = torch.where(there, first[:, None] + j, 0)
        k, v = (st[x][at].float().permute(0, 2, 1, 3) for x in "kv")  # [B, H, top, D]
        rows = max(1, min(top, (1 << 27) // (B * Hq * top)))          # query rows at a time
        for r in range(0, top, rows):
            i = j[r:r + rows]
            to = min(top, r + rows) if c["causal"] else top           # positions that these rows see
            q = st["q"][at[:, r:r + rows]].float().view(B, len(i), H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * len(i), D)
            s = torch.matmul(q, k[:, :, :to].transpose(-1, -2)) / math.sqrt(D)
            dead = ~there[:, None, None, None, :to]
            if c["causal"]:
                dead = dead | (j[:to] > i[:, None])
            p = _plain_softmax(s.view(B, H, G, len(i), to), dead)
            o = torch.matmul(p.view(B, H, G * len(i), to), v[:, :, :to]).view(B, H, G, len(i), D)
            o = o.permute(0, 3, 1, 2, 4).reshape(B, len(i), Hq, D).to(BF16)
            live = there[:, r:r + rows]
            out[at[:, r:r + rows][live]] = o[live]
    return out


def _plain_paged(st):
    c, q, ctx, rows = st["case"], st["q"].float(), st["ctx"], st["rows"]
    R, n_q, Hq, D = q.shape
    H, G = c["H"], Hq // c["H"]
    kv = st["pages"][rows.clamp(min=0)].float()                       # [R, pages, 2, H, block, D]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, R, H, -1, D)
    q = q.view(R, n_q, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, n_q * G, D)
    s = torch.matmul(q, kv[0].transpose(-1, -2)) / math.sqrt(D)
    limit = ctx[:, None] - n_q + 1 + torch.arange(n_q, device=DEV)    # [R, n_q]
    dead = (torch.arange(s.shape[-1], device=DEV) >= limit[..., None]).repeat_interleave(G, 1)[:, None]
    o = torch.matmul(_plain_softmax(s, dead), kv[1])
    return o.view(R, H, n_q, G, D).permute(0, 2, 1, 3, 4).reshape(R, n_q, Hq, D).to(BF16)


_RUN = {"rotary": _plain_rotary, "prompt": _plain_prompt, "paged": _plain_paged}
_RUN_OWN = {"rotary": _own_rotary, "prompt": _own_prompt, "paged": _own_paged}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------

def work(case):
    op, lens = case["op"], _lengths(case)
    H, Hq, D = case["H"], case["Hq"], case["D"]
    if op == "rotary":
        n = sum(_spans(case, lens)[1])
        e = 2 if case["src"] == "bf16" else 4
        if case["mode"] == "apply":
            return {"bytes": n * (2 * e * D * (Hq + H) + 4), "flops": 3 * n * (Hq + H) * case["rot"]}
        # q, k and v in; q (and a prompt's k) out, K and V into the cache; slots and positions
        back = Hq if case["mode"] == "step" else Hq + H
        return {"bytes": n * (D * (e * (Hq + 2 * H + back) + 4 * H) + 12), "flops": 3 * n * (Hq + H) * case["rot"]}
    if op == "prompt":
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return {"bytes": 4 * D * (Hq + H) * sum(lens), "flops": 4 * D * Hq * pairs}
    W, n_q, gen, block = case["W"], case["n_q"], case["gen"], case["block"]
    # every distinct cached position once: a page that several beams of a sentence share counts once
    ids = _beam_pages(case, lens, 0)[0]
    cached = 0
    for b, p in enumerate(lens):
        named = {(i, j) for r in ids[b * W:(b + 1) * W] for j, i in enumerate(r)}
        cached += sum(max(0, min(block, p + gen - j * block)) for _, j in named)
    pairs = sum(max(0, p + gen - i) for p in lens for i in range(n_q)) * W * Hq
    return {"bytes": 4 * H * D * cached + 4 * len(lens) * W * n_q * Hq * D, "flops": 4 * D * pairs}


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


def _exact_rotary(case, seed):
    st = _plain_state(case, seed)
    rot, pos = case["rot"], st["pos"].double()
    p = _SCALING[case["scaling"]]
    q, k = st["q"].double(), st["k"].double()
    new_q, new_k = q.clone(), k.clone()
    for i in range(rot // 2):
        if case["scaling"] == "base":
            f = (_BASE["base"] * p["factor"] ** (rot / (rot - 2))) ** (-2.0 * i / rot)
        else:
            f = _BASE[case["scaling"]] ** (-2.0 * i / rot)
        if case["scaling"] == "linear":
            f /= p["factor"]
        if case["scaling"] == "parts":
            turns = p["original"] * f / (2.0 * math.pi)
            if turns < p["low"]:
                f /= p["factor"]
            elif turns <= p["high"]:
                x = (turns - p["low"]) / (p["high"] - p["low"])
                f = (1.0 - x) * f / p["factor"] + x * f
        amp = p.get("amplitude", 1.0)
        c, s = (torch.cos(pos * f) * amp)[:, None], (torch.sin(pos * f) * amp)[:, None]
        a, b = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        for x, y in ((q, new_q), (k, new_k)):
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., a] * s + x[..., b] * c
    if case["mode"] == "apply":
        return [new_q, new_k]
    pool = st["pool"].double()
    at = st["slots"]
    pool[at // case["block"], 0, 0, :, at % case["block"]] = new_k
    pool[at // case["block"], 0, 1, :, at % case["block"]] = st["v"].double()
    return [new_q, pool] if case["mode"] == "step" else [new_q, new_k, pool]


def _softmax_rows64(q, k, v, scale, valid):
    """softmax(scale q k^T) v over the positions below valid[i] of each query i, in 64 bits; zeros where there are none."""
    s = (q @ k.T) * scale
    keep = torch.arange(k.shape[0], device=q.device)[None, :] < valid[:, None]
    s = torch.where(keep, s, -math.inf)
    top = s.max(dim=1, keepdim=True).values.clamp(min=-1e300)
    p = torch.where(keep, torch.exp(s - top), 0.0)
    z = p.sum(dim=1, keepdim=True)
    return torch.where(z > 0, (p @ v) / z.clamp(min=1e-300), 0.0)


def _exact_prompt(case, seed):
    # 64-bit products at about 1 TFLOP/s, and some 50 us a launch for the many small ones
    H, Hq, D, lens = case["H"], case["Hq"], case["D"], _lengths(case)
    if 4 * D * Hq * sum(n * n for n in lens) > 8e12 or len(lens) * Hq * 5e-4 > 15:
        return None
    st = _plain_state(case, seed)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for a, n in zip(st["starts"], st["lens"]):
        for h in range(Hq):
            k, v = (st[x][a:a + n, h // (Hq // H)].double() for x in "kv")
            for r in range(0, n, 2048):
                z = min(n, r + 2048)
                to = z if case["causal"] else n
                valid = torch.arange(r, z, device=DEV) + 1 if case["causal"] else torch.full((z - r,), n, device=DEV)
                out[a + r:a + z, h] = _softmax_rows64(st["q"][a + r:a + z, h].double(), k[:to], v[:to], D ** -0.5, valid)
    return out


def _exact_paged(case, seed):
    st = _plain_state(case, seed)
    q, ctx, rows = st["q"].double(), st["ctx"].tolist(), st["rows"].tolist()
    H, n_q, Hq, D = case["H"], case["n_q"], case["Hq"], case["D"]
    G = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    step = torch.arange(n_q, device=DEV).repeat_interleave(G)
    if q.shape[0] * H > 4096:
        return None
    for r in range(q.shape[0]):
        ids = [i for i in rows[r] if i >= 0]
        if not ids:
            continue
        vals = st["pages"][torch.tensor(ids, device=DEV)].double()    # [pages, 2, H, block, D]
        for h in range(H):
            mine = q[r, :, h * G:(h + 1) * G].reshape(n_q * G, D)
            o = _softmax_rows64(mine, vals[:, 0, h].reshape(-1, D), vals[:, 1, h].reshape(-1, D), D ** -0.5,
                                ctx[r] - n_q + 1 + step)
            out[r, :, h * G:(h + 1) * G] = o.view(n_q, G, D)
    return out


def exact(case, seed):
    return {"rotary": _exact_rotary, "prompt": _exact_prompt, "paged": _exact_paged}[case["op"]](case, seed)
