"""Measured cases of the operators around ring attention and the 4-bit cache.

* ``rope``: root-mean-square norms of queries and keys for each head, and the
  position rotation, in one pass (before ring attention, or before a cache step);
* ``rope_bwd``: its gradients, for the projections and for the norms' weights;
* ``weights``: the attention weight that each cached token receives from a
  step's query rows, accumulated over the query heads;
* ``evict``: for every request over its budget, the tokens with the smallest
  weights are dropped: which rows move where, the pages given back, and the
  move of the rows itself.

``run`` computes each in plain torch operations (``own`` false) or with the
framework's kernels (``own`` true); ``exact`` gives the same outputs from the
definition in float64.

The cache holds groups of 16 elements with a scale of 5 exponent and 3 mantissa
bits (bias 15, no sign: the byte shifted left by 7 is an fp16 number); an
element is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 16
EPS = 1e-6


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 requests somewhere in long contexts: slices of a fused projection, latency counts
        {"name": "rope-decode-64", "op": "rope", "T": 64, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "inter": False,
         "norm": True, "base": 500000.0, "pos": "far"},
        # a 32K prompt or training batch of packed documents before its ring attention
        {"name": "rope-docs-32k", "op": "rope", "T": 32768, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "inter": False,
         "norm": True, "base": 500000.0, "pos": "docs"},
        # the tiny two-head shape: 512 tokens
        {"name": "rope-bwd-tiny", "op": "rope_bwd", "T": 512, "Hq": 2, "Hkv": 2, "d": 64, "rot": 64, "inter": True,
         "norm": True, "base": 10000.0, "pos": "one"},
        # the packed variable-length training batch
        {"name": "rope-bwd-docs-64k", "op": "rope_bwd", "T": 65536, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "inter": False, "norm": True, "base": 500000.0, "pos": "docs"},
        # head_dim 256, a quarter of it rotated, an odd number of tokens
        {"name": "rope-bwd-d256", "op": "rope_bwd", "T": 30011, "Hq": 16, "Hkv": 8, "d": 256, "rot": 64,
         "inter": False, "norm": True, "base": 10000.0, "pos": "one"},
        # one token over a short cache, two heads: latency
        {"name": "weights-tiny", "op": "weights", "lens": "512", "qlens": "1", "Hq": 2, "Hkv": 2, "d": 64, "page": 16},
        # one token each of 128 requests with lognormal lengths
        {"name": "weights-ragged-128", "op": "weights", "lens": "lognormal:128", "qlens": "1", "Hq": 32, "Hkv": 8,
         "d": 128, "page": 64},
        # the last 64 tokens of a 32K prompt look back over it, before most of it is dropped
        {"name": "weights-window-32k", "op": "weights", "lens": "32768", "qlens": "64", "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64},
        # the next 1024 tokens of a prompt over the 32K already cached
        {"name": "weights-chunk-1k-32k", "op": "weights", "lens": "33792", "qlens": "1024", "Hq": 32, "Hkv": 8,
         "d": 128, "page": 64},
        # a small batch of short requests, two of them over their budget
        {"name": "evict-4x500", "op": "evict", "lens": "530,411,577,512", "budget": 512, "slack": 16, "recent": 16,
         "sinks": 4, "Hkv": 2, "d": 64, "page": 16, "moves": 66},
        # a serving step: 64 requests that grow from their budget of 4096 tokens, those 64 tokens over it are cut
        {"name": "evict-64x4k", "op": "evict", "lens": "over:64:65", "budget": 4096, "slack": 64, "recent": 64,
         "sinks": 4, "Hkv": 8, "d": 128, "page": 64, "moves": 65},
        # a 128K prompt cut to 8192 tokens before its answer is generated
        {"name": "evict-128k-8k", "op": "evict", "lens": "131072", "budget": 8192, "slack": 64, "recent": 64,
         "sinks": 4, "Hkv": 8, "d": 128, "page": 64, "moves": 8192},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "rope_bwd", "rope_bwd", "weights", "weights", "weights", "evict", "evict"])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op in ("rope", "rope_bwd"):
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 3, 4, 7, 8])
        cap = 32768 * 40 * 128 // (Hkv * (G + 1) * d)
        return {"op": op, "T": _log_int(rng, 1, min(cap, 131072)), "Hq": Hkv * G, "Hkv": Hkv, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4]), "inter": rng.random() < 0.4, "norm": rng.random() < 0.85,
                "base": rng.choice([10000.0, 500000.0, 1000000.0]), "pos": rng.choice(["one", "docs", "far"])}
    if op == "weights":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        kind = rng.choice(["decode", "decode", "verify", "window", "chunk"])
        most = {"decode": 1, "verify": 8, "window": 64, "chunk": 700}[kind]
        R = _log_int(rng, 1, {"decode": 128, "verify": 128, "window": 16, "chunk": 4}[kind])
        # cached elements and query-key pairs stay below those of the largest listed cases
        tokens = 128 * 4096 * 1024 // max(1, R) // (Hkv * d)
        pairs = 32 * 128 * 1024 * 32768 // (Hkv * G * d)
        lens, qlens = [], []
        for _ in range(R):
            n = 1 if kind == "decode" else _log_int(rng, 1, most)
            L = _log_int(rng, 1, max(8, min(131072, tokens, pairs // max(1, n * R))))
            lens.append(L)
            qlens.append(min(n, L))
        return {"op": op, "lens": ",".join(map(str, lens)), "qlens": ",".join(map(str, qlens)), "Hq": Hkv * G,
                "Hkv": Hkv, "d": d, "page": page}
    Hkv = rng.choice([1, 2, 4, 8])
    R = _log_int(rng, 1, 128)
    most = max(64, min(131072, 256 * 1024 * 1024 // (R * Hkv * d)))
    budget = _log_int(rng, 16, max(16, most // 2))
    recent = rng.randint(0, min(64, budget // 2))
    sinks = rng.randint(0, min(8, budget - recent))
    slack = max(recent, rng.randint(0, 128))
    lens = [max(1, min(most + slack, int(budget * math.exp(rng.uniform(-0.3, 1.2))) + rng.randint(0, slack + 1)))
            for _ in range(R)]
    return {"op": op, "lens": ",".join(map(str, lens)), "budget": budget, "slack": slack, "recent": recent,
            "sinks": sinks, "Hkv": Hkv, "d": d, "page": page, "moves": min(budget, max(1, max(lens) - budget))}


def _lens(case):
    s = case["lens"]
    if s.startswith("lognormal:"):
        n = int(s.split(":")[1])
        g = torch.Generator().manual_seed(1234)
        x = torch.exp(7.5 + 1.2 * torch.randn(n, generator=g, dtype=torch.float64))
        return [int(v) for v in x.clamp(128, 32768)]
    if s.startswith("over:"):
        # requests at every stage between their budget and the length at which they are cut, a quarter of them there
        n, most = (int(x) for x in s.split(":")[1:])
        return [case["budget"] + (most if i % 4 == 0 else i * 7 % most) for i in range(n)]
    return [int(v) for v in s.split(",")]


def _qlens(case):
    q = [int(v) for v in case["qlens"].split(",")]
    return q * len(_lens(case)) if len(q) == 1 else q


# ---------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 29)


def _rows(g, *shape):
    """Queries, keys or values as a projection makes them: normal, with a few strong channels."""
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
    gain = torch.exp(0.5 * torch.randn(shape[-2], shape[-1], generator=g, device=DEV))
    return (x * gain).to(torch.bfloat16)


def _positions(g, case):
    T, kind = case["T"], case["pos"]
    t = torch.arange(T, device=DEV)
    if kind == "one":                     # one document
        return t.int()
    if kind == "far":                     # single tokens, each somewhere in a context of up to a million
        return torch.randint(0, 1 << 20, (T,), generator=g, device=DEV).int()
    # packed documents of about 1600 tokens
    first = torch.rand(T, generator=g, device=DEV) < 1.0 / 1600
    first[0] = True
    start = torch.cummax(torch.where(first, t, torch.zeros_like(t)), 0)[0]
    return (t - start).int()


def _draw_rope(case, seed):
    g = _gen(seed)
    T, Hq, Hkv, d = case["T"], case["Hq"], case["Hkv"], case["d"]
    # slices of one projection's output (queries, keys, values): rows further apart than they are long
    qkv = torch.cat([_rows(g, T, Hq, d), _rows(g, T, 2 * Hkv, d)], dim=1)
    st = {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "pos": _positions(g, case), "wq": None, "wk": None}
    if case["norm"]:
        st["wq"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
        st["wk"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    if case["op"] == "rope_bwd":
        st["gq"] = torch.randn(T, Hq, d, generator=g, device=DEV).to(torch.bfloat16)
        st["gk"] = torch.randn(T, Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    return st


def _draw_pages(g, lens, P):
    """Block table over a pool with some spare pages, in random order; pages of the pool; the spare ones."""
    held = [(n + P - 1) // P for n in lens]
    W, total = max(held) + 1, sum(held)
    N = total + 3
    ids = torch.randperm(N, generator=g, device=DEV).int()
    per = torch.tensor(held, device=DEV)
    first = torch.cumsum(per, 0) - per
    j = torch.arange(W, device=DEV)
    table = torch.where(j < per[:, None], ids[(first[:, None] + j).clamp(max=N - 1)], torch.full((), -1, dtype=torch.int32, device=DEV))
    return table, N, ids[total:]


def _slots_of(table, P, lens):
    """Slots of every cached token, request by request."""
    per = torch.tensor(lens, device=DEV)
    req = torch.repeat_interleave(torch.arange(len(lens), device=DEV), per)
    pos = torch.arange(sum(lens), device=DEV) - torch.repeat_interleave(torch.cumsum(per, 0) - per, per)
    return table[req, pos // P].long() * P + pos % P


def _draw_weights(case, seed):
    g = _gen(seed)
    lens, qlens, P = _lens(case), _qlens(case), case["page"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    table, N, _ = _draw_pages(g, lens, P)
    T = sum(lens)
    k, v = _rows(g, T, Hkv, d), _rows(g, T, Hkv, d)
    cu_k, cu_q = [0], [0]
    for n, m in zip(lens, qlens):
        cu_k.append(cu_k[-1] + n)
        cu_q.append(cu_q[-1] + m)
    q = torch.randn(cu_q[-1], Hq, d, generator=g, device=DEV).to(torch.bfloat16)
    return {"q": q, "k": k, "v": v, "slots": _slots_of(table, P, lens), "table": table, "N": N, "lens": lens,
            "qlens": qlens, "cu_k": cu_k, "cu_q": cu_q, "lens_t": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "cu_q_t": torch.tensor(cu_q, dtype=torch.int32, device=DEV)}


def _draw_lse(case, a):
    """The log-sum-exp of the rows' attention over what the cache holds, as the attention call gave it (fp32)."""
    q, P = a["q"], case["page"]
    T, Hq, d = q.shape
    Hkv = case["Hkv"]
    lse = torch.empty(Hq, T, dtype=torch.float32, device=DEV)
    for r, (L, n) in enumerate(zip(a["lens"], a["qlens"])):
        b, c = a["cu_q"][r], a["cu_k"][r]
        kk = _plain_values(*_plain_round(a["k"][c:c + L]))                            # [L, Hkv, d]
        qq = q[b:b + n].float().reshape(n, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
        s = torch.matmul(qq, kk.permute(1, 2, 0)).reshape(Hq, n, L) / math.sqrt(d)
        hide = torch.arange(L, device=DEV) > L - n + torch.arange(n, device=DEV)[:, None]
        lse[:, b:b + n] = torch.logsumexp(s.masked_fill_(hide, -math.inf), -1)
    return lse


def _draw_evict(case, seed):
    g = _gen(seed)
    lens, P = _lens(case), case["page"]
    table, N, spare = _draw_pages(g, lens, P)
    T = sum(lens)
    k, v = _rows(g, T, case["Hkv"], case["d"]), _rows(g, T, case["Hkv"], case["d"])
    # accumulated weights: a few heavy tokens, many light ones
    slots = _slots_of(table, P, lens)
    weights = torch.zeros(N * P, device=DEV)
    weights[slots] = torch.exp(2.0 * torch.randn(T, generator=g, device=DEV))
    free = torch.full((N,), -1, dtype=torch.int32, device=DEV)
    free[:len(spare)] = spare
    return {"k": k, "v": v, "slots": slots, "table": table, "N": N, "weights": weights, "free": free,
            "count": torch.tensor([len(spare)], dtype=torch.int32, device=DEV), "lens": lens,
            "lens_t": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "budgets": torch.full((len(lens),), case["budget"], dtype=torch.int32, device=DEV)}


def prepare(case, seed):
    st = {"case": dict(case), "op": case["op"]}
    if own:
        import context_ring_attention_step_gb300 as ra
        st["ra"] = ra
    if case["op"] in ("rope", "rope_bwd"):
        st.update(_draw_rope(case, seed))
        if own:
            st["rotary"] = ra.Rotary(case["d"], case["rot"], base=case["base"], interleaved=case["inter"], device=DEV)
            st["out"] = tuple(torch.empty(case["T"], case[h], case["d"], dtype=torch.bfloat16, device=DEV)
                              for h in ("Hq", "Hkv"))
            if case["op"] == "rope_bwd":
                st["ws"] = ra.qk_norm_rope_workspace(case["d"], DEV)
        return st
    a = _draw_weights(case, seed) if case["op"] == "weights" else _draw_evict(case, seed)
    k, v, slots = a.pop("k"), a.pop("v"), a.pop("slots")
    if case["op"] == "weights":
        st["lse"] = _draw_lse(case, {**a, "k": k})
        st["weights"] = torch.zeros(a["N"] * case["page"], device=DEV)
        st["index"] = torch.arange(max(a["lens"]), device=DEV)
        # the last key that each query row sees
        st["limits"] = torch.cat([L - n + torch.arange(n, device=DEV) for L, n in zip(a["lens"], a["qlens"])])
    st.update(a)
    if own:
        st["cache"] = ra.Kv4Cache(a["N"], case["page"], case["Hkv"], case["d"], DEV)
        ra.kv4_store(st["cache"], k, v, slots)
        if case["op"] == "weights":
            st["ws"] = ra.kv4_attention_workspace(st["cache"], a["cu_q"][-1], case["Hq"], max(a["qlens"]))
        else:
            st["ws"] = ra.kv4_evict_workspace(len(a["lens"]), DEV)
            st["out"] = ra.kv4_evict_out(len(a["lens"]), case["moves"], DEV)
            st["rows"] = tuple(torch.empty(len(a["lens"]) * case["moves"], case["Hkv"], case["d"],
                                           dtype=torch.bfloat16, device=DEV) for _ in range(2))
    else:
        st["cache"] = _plain_cache(a["N"] * case["page"] + 1, case["Hkv"], case["d"])   # and one slot for no row
        _plain_store(st["cache"], k, v, slots)
    return st


# ---------------------------------------------------------------------- plain forms

def _plain_cache(slots, Hkv, d):
    """Codes two to a byte and scale bytes, one row a slot."""
    return {n: torch.zeros(slots, Hkv, w, dtype=torch.uint8, device=DEV)
            for n, w in (("kc", d // 2), ("ks", d // GROUP), ("vc", d // 2), ("vs", d // GROUP))}


def _plain_round(x):
    """(codes packed two to a byte, scale bytes) of rows [T, H, d]."""
    T, H, d = x.shape
    x = x.float().reshape(T, H, d // GROUP, GROUP)
    s = (x.abs().amax(-1) / 6.0).clamp(max=10240.0)
    e = torch.frexp(s)[1].clamp(min=-13) - 1                      # s in [2^e, 2^(e+1)), e >= -14
    quantum = torch.ldexp(torch.ones_like(s), e - 3)
    s = torch.round(s / quantum) * quantum
    sbyte = (s.half().view(torch.int16) >> 7).to(torch.uint8)
    y = torch.where((s > 0).unsqueeze(-1), x / s.unsqueeze(-1), torch.zeros_like(x))
    a = y.abs()
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    a = a.clamp(max=6.0)
    mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (mag | ((y < 0).to(torch.uint8) << 3)).reshape(T, H, d)
    return code[..., 0::2] | (code[..., 1::2] << 4), sbyte


def _plain_values(codes, sbyte):
    """fp32 values of packed codes [..., d/2] and scale bytes [..., d/16]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    s = (sbyte.to(torch.int16) << 7).view(torch.float16).float()
    return (lut[c.int()].unflatten(-1, (-1, GROUP)) * s.unsqueeze(-1)).flatten(-2)


def _plain_store(cache, k, v, slots):
    for x, c, s in ((k, "kc", "ks"), (v, "vc", "vs")):
        codes, sb = _plain_round(x)
        cache[c][slots] = codes
        cache[s][slots] = sb


def _plain_angles(case, pos):
    """cos and sin [T, 1, rot / 2] of the positions' angles, taken in 64 bits: far positions have large angles."""
    rot = case["rot"]
    freq = case["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = (pos.double()[:, None] * freq)[:, None]
    return torch.cos(a).float(), torch.sin(a).float()


def _plain_turn(case, x, cos, sin):
    """Rotate the first rot elements of rows [T, H, d] (fp32)."""
    rot = case["rot"]
    if case["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope(case, x, w, cos, sin):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _plain_turn(case, x, cos, sin).to(torch.bfloat16)


def _plain_rope_bwd(case, x, w, g, cos, sin):
    h = _plain_turn(case, g.float(), cos, -sin)
    if w is None:
        return h.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    dw = (h * n).sum((0, 1))
    h = h * w
    return (r * (h - n * (h * n).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _plain_weights(st):
    q, case = st["q"], st["case"]
    T, Hq, d = q.shape
    Hkv, P = case["Hkv"], case["page"]
    slots = _slots_of(st["table"], P, st["lens"])
    keys = _plain_values(st["cache"]["kc"][slots], st["cache"]["ks"][slots]).permute(1, 2, 0)   # [Hkv, d, all tokens]
    rows = q.float().reshape(T, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3) * (1.0 / math.sqrt(d))   # [Hkv, G, T, d]
    sums = []
    for r, (L, n) in enumerate(zip(st["lens"], st["qlens"])):
        b, c = st["cu_q"][r], st["cu_k"][r]
        s = torch.matmul(rows[:, :, b:b + n].reshape(Hkv, -1, d), keys[:, :, c:c + L]).reshape(Hq, n, L)
        p = torch.exp(s - st["lse"][:, b:b + n, None])
        sums.append((p.sum(0) * (st["index"][:L] <= st["limits"][b:b + n, None])).sum(0))
    out = torch.zeros_like(st["weights"])
    out[slots] = torch.cat(sums)
    return out


def _plain_evict(st):
    case = st["case"]
    P, B, M = case["page"], case["budget"], case["moves"]
    L, table, w = st["lens_t"].long(), st["table"].long(), st["weights"]
    R = L.numel()
    top = max(st["lens"])
    i = torch.arange(top, device=DEV)
    live = i < L[:, None]
    slots = torch.where(live, table[:, i // P] * P + i % P, torch.full((), -1, device=DEV))
    cut = L > B + case["slack"]
    after = torch.where(cut, torch.full_like(L, B), L)
    # keys in order: protected tokens first, then by weight; a stable sort puts the lowest index first among equals
    key = torch.where(live, w[slots.clamp(min=0)], torch.full((), -1.0, device=DEV))
    safe = live & ((i < case["sinks"]) | (i >= L[:, None] - case["recent"]))
    order = torch.sort(torch.where(safe, torch.full((), math.inf, device=DEV), key), dim=1, descending=True,
                       stable=True)[1]
    kept = torch.zeros(R, top, dtype=torch.bool, device=DEV)
    kept.scatter_(1, order[:, :B], True)
    kept &= live
    hole = cut[:, None] & ~kept & (i < B)
    mover = cut[:, None] & kept & (i >= B)
    lists = []
    pad = max(M, top) + 1
    for m in (mover, hole):
        rank = torch.where(m, torch.cumsum(m.long(), 1) - 1, torch.full_like(order, pad - 1))
        lists.append(torch.full((R, pad), -1, device=DEV).scatter_(1, rank, torch.where(m, slots, -1))[:, :M].contiguous())
    # pages behind the new length go back, in request order, page order
    held, need = (L + P - 1) // P, (after + P - 1) // P
    back = held - need
    j = torch.arange(table.shape[1], device=DEV)
    put = (j >= need[:, None]) & (j < held[:, None])
    place = st["count"].long() + (torch.cumsum(back, 0) - back)[:, None] + j - need[:, None]
    free = torch.cat([st["free"], st["free"].new_zeros(1)])
    free.scatter_(0, torch.where(put, place, torch.full_like(place, free.numel() - 1)).flatten(), st["table"].flatten())
    # the moves themselves, and the rows that now lie there
    src, dst = (x.flatten() for x in lists)
    go = dst >= 0
    cache = st["cache"]
    at = torch.where(go, dst, cache["kc"].shape[0] - 1)
    rows = []
    for n in ("kc", "ks", "vc", "vs"):
        new = cache[n][src.clamp(min=0)]
        cache[n].index_copy_(0, at, new)
        rows.append(new)
    k, v = (torch.where(go[:, None, None], _plain_values(c, s), torch.zeros((), device=DEV)).to(torch.bfloat16)
            for c, s in (rows[:2], rows[2:]))
    return (after.int(), (L - after).int(), lists[0], lists[1], (st["count"] + back.sum()).int(), free[:-1], k, v)


# ---------------------------------------------------------------------- one pass

def run(st):
    op, case = st["op"], st["case"]
    if own:
        ra = st["ra"]
        eps = EPS if case.get("norm") else None
        if op == "rope":
            return ra.qk_norm_rope_fwd(st["q"], st["k"], st["pos"], st["rotary"], st["wq"], st["wk"], eps=eps,
                                       out=st["out"])
        if op == "rope_bwd":
            return ra.qk_norm_rope_bwd(st["q"], st["k"], st["gq"], st["gk"], st["pos"], st["rotary"], st["wq"],
                                       st["wk"], eps=eps, workspace=st["ws"], out=st["out"])
        if op == "weights":
            # the accumulators of all tokens begin with this step
            ra.kv4_weights(st["q"], st["cache"], st["table"], st["lens_t"], st["cu_q_t"], st["lse"], st["weights"],
                           new_lens=st["lens_t"], max_q_len=max(st["qlens"]), workspace=st["ws"])
            return st["weights"]
        e = ra.kv4_evict(st["weights"], st["table"], st["lens_t"], st["budgets"], case["page"], case["moves"],
                         slack=case["slack"], recent=case["recent"], sinks=case["sinks"], free_pages=st["free"],
                         free_count=st["count"], workspace=st["ws"], out=st["out"])
        ra.kv4_move(st["cache"], e.src_slots, e.dst_slots)
        k, v = ra.kv4_load(st["cache"], e.dst_slots.view(-1), out=st["rows"])
        return e.kv_lens, e.dropped, e.src_slots, e.dst_slots, e.free_count, st["free"], k, v
    if op == "rope":
        cos, sin = _plain_angles(case, st["pos"])
        return _plain_rope(case, st["q"], st["wq"], cos, sin), _plain_rope(case, st["k"], st["wk"], cos, sin)
    if op == "rope_bwd":
        cos, sin = _plain_angles(case, st["pos"])
        dq, dwq = _plain_rope_bwd(case, st["q"], st["wq"], st["gq"], cos, sin)
        dk, dwk = _plain_rope_bwd(case, st["k"], st["wk"], st["gk"], cos, sin)
        return dq, dk, dwq, dwk
    if op == "weights":
        return _plain_weights(st)
    return _plain_evict(st)


def work(case):
    if case["op"] in ("rope", "rope_bwd"):
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["d"]
        # rows in and out (backward: rows and their gradients in, gradients out), positions, frequencies, weights
        side = 4 * case["T"] + 4 * case["rot"] + (8 * case["d"] if case["norm"] else 0)
        if case["op"] == "rope":
            return {"bytes": 4 * n + side, "flops": 8 * n}
        return {"bytes": (6 if case["norm"] else 4) * n + side + (8 * case["d"] if case["norm"] else 0), "flops": 16 * n}
    lens = _lens(case)
    Hkv, d = case["Hkv"], case["d"]
    pages = 4 * sum(-(-L // case["page"]) for L in lens)
    if case["op"] == "weights":
        qlens = _qlens(case)
        pairs = sum(n * L - n * (n - 1) // 2 for L, n in zip(lens, qlens))
        return {"bytes": sum(lens) * (Hkv * d * 9 // 16 + 4) + sum(qlens) * case["Hq"] * (2 * d + 4) + pages,
                "flops": 2 * d * case["Hq"] * pairs}
    B, M = case["budget"], case["moves"]
    cut = [L for L in lens if L > B + case["slack"]]
    # weights of the requests that are cut; lists of moves; the rows that move (about budget of length of those behind
    # the budget), and all listed rows read back as bf16
    moved = sum(B * (L - B) // L for L in cut)
    return {"bytes": 4 * sum(cut) + 16 * len(lens) * M + pages + moved * Hkv * d * 9 // 8 * 3 + len(lens) * M * Hkv * d * 4,
            "flops": 0}


# ---------------------------------------------------------------------- float64 definitions

def _exact_rope(case, x, pos, w):
    """Rows of one head [T, d] in float64: norm, then pairs as complex numbers times exp(i angle)."""
    rot = case["rot"]
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    a = torch.outer(pos.double(), torch.exp(-2 * i / rot * math.log(case["base"])))
    pairs = x[:, :rot].unflatten(-1, (-1, 2)) if case["inter"] else x[:, :rot].unflatten(-1, (2, -1)).transpose(1, 2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(a), a))
    return torch.cat([z.flatten(1) if case["inter"] else z.transpose(1, 2).flatten(1), x[:, rot:]], dim=-1)


def _exact_values(x):
    """What the cache holds for rows x, from the nearest values of the two formats."""
    x = x.double().unflatten(-1, (-1, GROUP))
    amax = x.abs().amax(-1, keepdim=True)
    # all scales: 0, the subnormals and the normal numbers up to 10240
    scales = torch.tensor([m * 2.0 ** -17 for m in range(8)]
                          + [(8 + m) * 2.0 ** (e - 3) for e in range(-14, 14) for m in range(8)
                             if (8 + m) * 2.0 ** (e - 3) <= 10240], dtype=torch.float64, device=x.device)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)

    def nearest(y, values):
        mid = (values[1:] + values[:-1]) / 2
        lo, hi = torch.searchsorted(mid, y, right=False), torch.searchsorted(mid, y, right=True)
        even = torch.where(lo % 2 == 0, lo, hi)                   # on a border: the even code
        return values[even]

    s = nearest(amax / 6.0, scales)
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    return (torch.sign(x) * nearest(y, grid) * s).flatten(-2)


def _exact_evict(case, seed):
    a = _draw_evict(case, seed)
    P, B, M, R = case["page"], case["budget"], case["moves"], len(a["lens"])
    table, free, count = a["table"].tolist(), a["free"].tolist(), int(a["count"])
    w = a["weights"].tolist()
    src, dst, where = [[-1] * M for _ in range(R)], [[-1] * M for _ in range(R)], torch.full((R, M), -1)
    after, base = [], 0
    for r, L in enumerate(a["lens"]):
        slot = [table[r][i // P] * P + i % P for i in range(L)]
        after.append(B if L > B + case["slack"] else L)
        if after[r] < L:
            last = L - case["recent"]
            ranked = sorted(range(case["sinks"], last), key=lambda i: (-w[slot[i]], i))
            kept = set(range(case["sinks"])) | set(range(last, L)) | set(ranked[:B - case["sinks"] - case["recent"]])
            holes = [i for i in range(B) if i not in kept]
            for m, (h, i) in enumerate(zip(holes, sorted(i for i in kept if i >= B))):
                src[r][m], dst[r][m], where[r, m] = slot[i], slot[h], base + i
            for j in range(-(-B // P), -(-L // P)):
                free[count] = table[r][j]
                count += 1
        base += L
    i32 = dict(dtype=torch.int32, device=DEV)
    lens = torch.tensor(a["lens"], **i32)
    after = torch.tensor(after, **i32)
    where = where.flatten().to(DEV)
    k, v = (torch.where((where >= 0)[:, None, None], _exact_values(x[where.clamp(min=0)]), 0.0).to(torch.bfloat16)
            for x in (a["k"], a["v"]))
    return (after, lens - after, torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV),
            torch.tensor([count], **i32), torch.tensor(free, **i32), k, v)


def exact(case, seed):
    if case["op"] in ("rope", "rope_bwd"):
        a = _draw_rope(case, seed)
        outs = []
        for x, w, g in ((a["q"], a["wq"], a.get("gq")), (a["k"], a["wk"], a.get("gk"))):
            w = None if w is None else w.double().requires_grad_(g is not None)
            rows = []
            for h in range(x.shape[1]):
                leaf = x[:, h].double().requires_grad_(g is not None)
                y = _exact_rope(case, leaf, a["pos"], w)
                if g is not None:
                    y.backward(g[:, h].double())
                rows.append(y if g is None else leaf.grad)
            outs.append((torch.stack(rows, dim=1), None if w is None else w.grad))
        (y, dwq), (z, dwk) = outs
        return (y, z) if case["op"] == "rope" else (y, z, dwq, dwk)
    if case["op"] == "evict":
        return _exact_evict(case, seed)
    a = _draw_weights(case, seed)
    lse = _draw_lse(case, a)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    out = torch.zeros(a["N"] * case["page"], dtype=torch.float64, device=DEV)
    for r, (L, n) in enumerate(zip(a["lens"], a["qlens"])):
        kb, qb = a["cu_k"][r], a["cu_q"][r]
        sums = torch.zeros(L, dtype=torch.float64, device=DEV)
        for h in range(Hkv):
            kk = _exact_values(a["k"][kb:kb + L, h])
            for i0 in range(0, n, 256):
                i1 = min(n, i0 + 256)
                qq = a["q"][qb + i0:qb + i1, h * G:(h + 1) * G].double().reshape(-1, d)
                x = (qq @ kk.t()).reshape(i1 - i0, G, L) / math.sqrt(d)
                x -= lse[h * G:(h + 1) * G, qb + i0:qb + i1].double().t().unsqueeze(-1)
                i = torch.arange(i0, i1, device=DEV).view(-1, 1, 1)
                x.masked_fill_(torch.arange(L, device=DEV) > L - n + i, -math.inf)
                sums += torch.exp(x).sum((0, 1))
        out[a["slots"][kb:kb + L]] = sums
    return out
