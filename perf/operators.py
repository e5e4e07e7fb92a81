"""Measured cases of the 4-bit key/value cache operators.

Four operators, as a serving loop next to ring attention uses them:

* ``tables``: from the requests' lengths, take and release pages and build the
  block table, the slot map and the positions of a step's new tokens;
* ``store``: round new key/value rows to 4 bits and put them into the pages
  (measured together with reading the rows back, which gives the values that
  the cache then holds);
* ``load``: read cached rows back as dense bf16 tensors;
* ``attn``: attention of packed query rows over the cache.

``run`` computes each in plain torch operations (``own`` false) or with the
framework's kernels (``own`` true); ``exact`` gives the same outputs from the
definition in float64.

The cache format: groups of 16 elements along head_dim share a scale of 5
exponent and 3 mantissa bits (bias 15, no sign: the byte shifted left by 7 is
an fp16 number); an element is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 16


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a served batch: 64 requests, one token each
        {"name": "tables-decode-64", "op": "tables", "R": 64, "page": 64, "W": 2048, "max_len": 32768,
         "prompts": 0, "max_prompt": 0, "released": 0, "slots": 64},
        # a step that also admits prompts and lets finished requests go
        {"name": "tables-admit-256", "op": "tables", "R": 256, "page": 64, "W": 2048, "max_len": 65536,
         "prompts": 32, "max_prompt": 8000, "released": 24, "slots": 262144},
        # the new rows of a decode step (Llama-3-8B attention shape: 8 key/value heads, head_dim 128)
        {"name": "store-decode-64", "op": "store", "T": 64, "Hkv": 8, "d": 128, "page": 64, "tokens": 65536},
        # the rows of a 32K prompt after its ring attention forward
        {"name": "store-prompt-32k", "op": "store", "T": 32768, "Hkv": 8, "d": 128, "page": 64, "tokens": 65536},
        # a short prefix of the tiny two-head shape
        {"name": "load-tiny", "op": "load", "T": 509, "Hkv": 2, "d": 64, "page": 16, "tokens": 4096},
        # a 128K prompt's keys and values back as dense tensors
        {"name": "load-128k", "op": "load", "T": 131072, "Hkv": 8, "d": 128, "page": 64, "tokens": 131072},
        # one token over a short cache, two heads: latency
        {"name": "attn-tiny", "op": "attn", "lens": "512", "qlens": "1", "Hq": 2, "Hkv": 2, "d": 64, "page": 16,
         "causal": True},
        # one token of one request at the 128K context
        {"name": "attn-1x128k", "op": "attn", "lens": "131072", "qlens": "1", "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "causal": True},
        # one token each of 128 requests with lognormal lengths (the packed variable-length workload's distribution)
        {"name": "attn-ragged-128", "op": "attn", "lens": "lognormal:128", "qlens": "1", "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "causal": True},
        # four drafted tokens and the last accepted one of 8 requests, checked at once
        {"name": "attn-verify-8x5", "op": "attn", "lens": "16111,15007,9973,20011,16384,12289,17000,8191",
         "qlens": "5", "Hq": 32, "Hkv": 8, "d": 128, "page": 32, "causal": True},
        # head_dim 256, groups of 8 query heads, four long requests
        {"name": "attn-4x64k-d256", "op": "attn", "lens": "65536,61001,50021,65001", "qlens": "1", "Hq": 16, "Hkv": 2,
         "d": 256, "page": 128, "causal": True},
        # the next 1024 tokens of a prompt over the 32K already cached
        {"name": "attn-chunk-1k-32k", "op": "attn", "lens": "33792", "qlens": "1024", "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "causal": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "store", "load", "attn", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        R = _log_int(rng, 1, 512)
        prompts = rng.randint(0, max(0, min(32, R // 4)))
        max_prompt = _log_int(rng, 1, 8000) if prompts else 0
        released = rng.randint(0, (R - prompts) // 4)
        need = R + prompts * max_prompt
        max_len = _log_int(rng, 16, 32768)
        return {"op": op, "R": R, "page": page, "W": (max_len + max_prompt) // page + 2, "max_len": max_len,
                "prompts": prompts, "max_prompt": max_prompt, "released": released,
                "slots": min(262144, need + rng.randint(0, max(1, need // 4)))}
    if op in ("store", "load"):
        d = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        cap = (33554432 if op == "store" else 134217728) // (Hkv * d)
        T = _log_int(rng, 1, min(cap, 131072))
        return {"op": op, "T": T, "Hkv": Hkv, "d": d, "page": page, "tokens": T + rng.randint(0, 4096)}
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    R = _log_int(rng, 1, 128)
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    qmax = {"decode": 1, "verify": 8, "chunk": 700}[kind]
    if kind == "chunk":
        R = min(R, 4)
    # cached elements and query-key pairs stay below those of the largest listed cases
    tokens = min(131072 * 8 * 128, 4 * 131072 * 1024 // max(1, R)) // (Hkv * d)
    pairs = 32 * 128 * 1024 * 30000 // (Hkv * G * d)
    lens, qlens = [], []
    for _ in range(R):
        n = 1 if kind == "decode" else _log_int(rng, 1, qmax)
        top = max(8, min(131072, tokens, pairs // max(1, n * R)))
        L = _log_int(rng, 1, top)
        lens.append(L)
        qlens.append(min(n, L))
    return {"op": op, "lens": ",".join(map(str, lens)), "qlens": ",".join(map(str, qlens)), "Hq": Hkv * G, "Hkv": Hkv,
            "d": d, "page": page, "causal": rng.random() < 0.85}


def _lens(case):
    s = case["lens"]
    if s.startswith("lognormal:"):
        n = int(s.split(":")[1])
        g = torch.Generator().manual_seed(1234)
        x = torch.exp(7.5 + 1.2 * torch.randn(n, generator=g, dtype=torch.float64))
        return [int(v) for v in x.clamp(128, 32768)]
    return [int(v) for v in s.split(",")]


def _qlens(case):
    q = [int(v) for v in case["qlens"].split(",")]
    return q * len(_lens(case)) if len(q) == 1 else q


# ---------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 17)


def _rows(g, *shape):
    """Keys or values as a model makes them: normal, with a few strong channels."""
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
    gain = torch.exp(0.5 * torch.randn(shape[-2], shape[-1], generator=g, device=DEV))
    return (x * gain).to(torch.bfloat16)


def _draw_tables(case, seed):
    """Lengths before the step, new lengths, block table and free pages."""
    g = torch.Generator().manual_seed(7919 * int(seed) + 5)
    R, P, W = case["R"], case["page"], case["W"]
    lens = torch.exp(torch.rand(R, generator=g, dtype=torch.float64) * math.log(case["max_len"])).long()
    new = torch.ones(R, dtype=torch.long)
    order = torch.randperm(R, generator=g)
    pr, rel = order[:case["prompts"]], order[case["prompts"]:case["prompts"] + case["released"]]
    if case["prompts"]:
        lens[pr] = 0
        new[pr] = 1 + torch.randint(0, case["max_prompt"], (len(pr),), generator=g)
    new[rel] = -1
    # the block table's rows hold as many tokens as W pages do
    lens = torch.minimum(lens, W * P - new.clamp(min=0))
    held = (lens + P - 1) // P
    # a pool that could hold every row of the table
    total, N = int(held.sum()), R * W
    spare = N - total
    ids = torch.randperm(N, generator=g)
    table = torch.full((R, W), -1, dtype=torch.int32)
    at = 0
    for r in range(R):
        n = int(held[r])
        table[r, :n] = ids[at:at + n].int()
        at += n
    free = torch.full((N,), -1, dtype=torch.int32)
    free[:spare] = ids[at:].int()
    return {"lens": lens.int(), "new": new.int(), "table": table, "free": free,
            "count": torch.tensor([spare], dtype=torch.int32)}


def _slots(g, T, tokens, page):
    """Slots of T cached tokens: the tokens of one request whose pages are in random order."""
    pages = (tokens + page - 1) // page
    table = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    return (table[t // page] * page + t % page).long(), pages


def _draw_rows(case, seed):
    g = _gen(seed)
    T, Hkv, d = case["T"], case["Hkv"], case["d"]
    slots, pages = _slots(g, T, case["tokens"], case["page"])
    # as a model has them: slices of one projection's output, rows further apart than they are long
    kv = torch.cat([_rows(g, T, Hkv, d), _rows(g, T, Hkv, d)], dim=1)
    return kv[:, :Hkv], kv[:, Hkv:], slots, pages


def _draw_attn(case, seed):
    g = _gen(seed)
    lens, qlens, P = _lens(case), _qlens(case), case["page"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    held = [(n + P - 1) // P for n in lens]
    W, total = max(held) + 1, sum(held)
    N = total + 3
    ids = torch.randperm(N, generator=g, device=DEV).int()
    table = torch.full((len(lens), W), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    T = sum(lens)
    k, v = _rows(g, T, Hkv, d), _rows(g, T, Hkv, d)
    cu_k = [0]
    for n in lens:
        cu_k.append(cu_k[-1] + n)
    pos = torch.cat([torch.arange(n, device=DEV) for n in lens])
    req = torch.cat([torch.full((n,), r, device=DEV) for r, n in enumerate(lens)])
    slots = table[req, pos // P].long() * P + pos % P
    cu_q = [0]
    for n in qlens:
        cu_q.append(cu_q[-1] + n)
    q = torch.randn(cu_q[-1], Hq, d, generator=g, device=DEV).to(torch.bfloat16)
    return {"q": q, "k": k, "v": v, "slots": slots, "table": table, "N": N, "lens": lens, "qlens": qlens,
            "cu_k": cu_k, "cu_q": cu_q,
            "lens_t": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "cu_q_t": torch.tensor(cu_q, dtype=torch.int32, device=DEV)}


def prepare(case, seed):
    st = {"case": dict(case), "op": case["op"]}
    if own:
        import context_ring_attention_step_gb300 as ra
        st["ra"] = ra
    if case["op"] == "tables":
        st.update({k: v.to(DEV) for k, v in _draw_tables(case, seed).items()})
        if own:
            st["out"] = ra.kv4_tables_out(case["R"], case["slots"], DEV)
        return st
    if case["op"] in ("store", "load"):
        k, v, slots, pages = _draw_rows(case, seed)
        st["slots"] = slots
        if own:
            st["cache"] = ra.Kv4Cache(pages, case["page"], case["Hkv"], case["d"], DEV)
            if case["op"] == "load":
                ra.kv4_store(st["cache"], k, v, slots)
        else:
            n = pages * case["page"]
            st["cache"] = _plain_cache(n, case["Hkv"], case["d"])
            if case["op"] == "load":
                _plain_store(st["cache"], k, v, slots)
        if case["op"] == "store":
            st["k"], st["v"] = k, v
        st["out"] = (torch.empty(case["T"], case["Hkv"], case["d"], dtype=torch.bfloat16, device=DEV),
                     torch.empty(case["T"], case["Hkv"], case["d"], dtype=torch.bfloat16, device=DEV))
        return st
    a = _draw_attn(case, seed)
    if own:
        st["cache"] = ra.Kv4Cache(a["N"], case["page"], case["Hkv"], case["d"], DEV)
        ra.kv4_store(st["cache"], a["k"], a["v"], a["slots"])
        T = a["cu_q"][-1]
        st["out"] = (torch.empty(T, case["Hq"], case["d"], dtype=torch.bfloat16, device=DEV),
                     torch.empty(case["Hq"], T, dtype=torch.float32, device=DEV))
        st["ws"] = ra.kv4_attention_workspace(st["cache"], T, case["Hq"], max(a["qlens"]))
    else:
        st["cache"] = _plain_cache(a["N"] * case["page"], case["Hkv"], case["d"])
        _plain_store(st["cache"], a["k"], a["v"], a["slots"])
    for name in ("q", "table", "lens", "qlens", "cu_q", "lens_t", "cu_q_t"):
        st[name] = a[name]
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
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    s = (torch.where(bad, torch.ones_like(amax), amax) / 6.0).clamp(max=10240.0)
    e = torch.frexp(s)[1].clamp(min=-13) - 1                      # s in [2^e, 2^(e+1)), e >= -14
    quantum = torch.ldexp(torch.ones_like(s), e - 3)
    s = torch.round(s / quantum) * quantum
    sbyte = (s.half().view(torch.int16) >> 7).to(torch.uint8)
    sbyte = torch.where(bad, torch.full_like(sbyte, 255), sbyte)
    y = torch.where((s > 0).unsqueeze(-1) & ~bad.unsqueeze(-1), x / s.unsqueeze(-1), torch.zeros_like(x))
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


def _plain_load(cache, slots):
    return tuple(_plain_values(cache[c][slots], cache[s][slots]).to(torch.bfloat16)
                 for c, s in (("kc", "ks"), ("vc", "vs")))


def _plain_tables(st):
    P, slots = st["case"]["page"], st["case"]["slots"]
    lens, new, table, free = st["lens"].long(), st["new"].long(), st["table"].clone(), st["free"].clone()
    R, W = table.shape
    held = (lens + P - 1) // P
    gone = new < 0
    take = new.clamp(min=0)
    after = torch.where(gone, torch.zeros_like(lens), lens + take)
    back = torch.where(gone, held, torch.zeros_like(held))
    need = torch.where(gone, torch.zeros_like(held), (after + P - 1) // P - held)
    j = torch.arange(W, device=DEV).unsqueeze(0)
    # released pages go back in request order, page order
    push = st["count"].long() + (torch.cumsum(back, 0) - back).unsqueeze(1) + j
    put = j < back.unsqueeze(1)
    free = torch.cat([free, free.new_zeros(1)])
    free.scatter_(0, torch.where(put, push, torch.full_like(push, free.numel() - 1)).flatten(), table.flatten())
    top = st["count"].long() + back.sum()
    # new pages come off the top, in request order, page order
    k = j - held.unsqueeze(1)
    got = (k >= 0) & (k < need.unsqueeze(1))
    pop = top - 1 - ((torch.cumsum(need, 0) - need).unsqueeze(1) + k)
    table = torch.where(got, free[torch.where(got, pop, torch.zeros_like(pop))], table)
    ends = torch.cumsum(take, 0)
    cu = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(slots, device=DEV)
    r = torch.searchsorted(ends, t, right=True).clamp(max=R - 1)
    live = t < ends[-1]
    pos = lens[r] + t - cu[r]
    page = table[r, torch.where(live, pos // P, torch.zeros_like(pos))].long()
    slot = torch.where(live, page * P + pos % P, torch.full_like(pos, -1))
    pos = torch.where(live, pos, torch.full_like(pos, -1))
    return (after.int(), cu.int(), slot, pos.int(), (top - need.sum()).int(), table, free[:-1])


def _plain_attn(st):
    q, case = st["q"], st["case"]
    T, Hq, d = q.shape
    Hkv, P = case["Hkv"], case["page"]
    G = Hq // Hkv
    o = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(Hq, T, dtype=torch.float32, device=DEV)
    scale = 1.0 / math.sqrt(d)
    for r, (L, n) in enumerate(zip(st["lens"], st["qlens"])):
        b = st["cu_q"][r]
        pos = torch.arange(L, device=DEV)
        slots = st["table"][r, pos // P].long() * P + pos % P
        limit = L - n + torch.arange(n, device=DEV) if case["causal"] else torch.full((n,), L - 1, device=DEV)
        for h in range(Hkv):
            kk = _plain_values(st["cache"]["kc"][slots, h], st["cache"]["ks"][slots, h])
            vv = _plain_values(st["cache"]["vc"][slots, h], st["cache"]["vs"][slots, h])
            qq = q[b:b + n, h * G:(h + 1) * G].float()
            s = torch.matmul(qq, kk.t()) * scale                                  # [n, G, L]
            s = torch.where((pos > limit.unsqueeze(1)).unsqueeze(1), torch.full((), -math.inf, device=DEV), s)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            z = p.sum(-1, keepdim=True)
            o[b:b + n, h * G:(h + 1) * G] = (torch.matmul(p, vv) / z).to(torch.bfloat16)
            lse[h * G:(h + 1) * G, b:b + n] = (m + torch.log(z)).squeeze(-1).t()
    return o, lse


# ---------------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        ra = st["ra"]
        if op == "tables":
            ra.kv4_tables(st["lens"], st["new"], st["table"], st["case"]["page"], st["case"]["slots"],
                          free_pages=st["free"], free_count=st["count"], out=st["out"])
            t = st["out"]
            return t.kv_lens, t.cu_new, t.slot_map, t.positions, t.free_count, st["table"], st["free"]
        if op == "store":
            ra.kv4_store(st["cache"], st["k"], st["v"], st["slots"])
            return ra.kv4_load(st["cache"], st["slots"], out=st["out"])
        if op == "load":
            return ra.kv4_load(st["cache"], st["slots"], out=st["out"])
        return ra.kv4_attention(st["q"], st["cache"], st["table"], st["lens_t"], st["cu_q_t"],
                                causal=st["case"]["causal"], max_q_len=max(st["qlens"]), workspace=st["ws"],
                                out=st["out"])
    if op == "tables":
        return _plain_tables(st)
    if op == "store":
        _plain_store(st["cache"], st["k"], st["v"], st["slots"])
        return _plain_load(st["cache"], st["slots"])
    if op == "load":
        return _plain_load(st["cache"], st["slots"])
    return _plain_attn(st)


def work(case):
    if case["op"] == "tables":
        # per request: two lengths in, a length and an offset out; per slot: a slot and a position out;
        # per new page: one free-list entry in, one table entry out
        pages = case["R"] // case["page"] + 1 + case["prompts"] * (case["max_prompt"] // 2 // case["page"] + 1)
        return {"bytes": 16 * case["R"] + 12 * case["slots"] + 8 * pages, "flops": 0}
    if case["op"] in ("store", "load"):
        n = case["T"] * case["Hkv"] * case["d"]
        dense, packed, slots = 4 * n, n * 9 // 8, 8 * case["T"]     # K and V: bf16, and 4.5 bits an element
        if case["op"] == "load":
            return {"bytes": dense + packed + slots, "flops": 2 * n}
        return {"bytes": 2 * (dense + packed + slots), "flops": 6 * n}
    lens, qlens = _lens(case), _qlens(case)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    T = sum(qlens)
    pairs = sum(n * L - (n * (n - 1) // 2 if case["causal"] else 0) for L, n in zip(lens, qlens))
    return {"bytes": sum(lens) * Hkv * d * 9 // 8 + 4 * T * Hq * d + 4 * Hq * T + 4 * sum(-(-L // case["page"]) for L in lens),
            "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------------- float64 definitions

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

    s = nearest(torch.nan_to_num(amax / 6.0, nan=0.0, posinf=0.0), scales)
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    v = torch.sign(x) * nearest(torch.nan_to_num(y), grid) * s
    v = torch.where(torch.isfinite(amax), v, torch.full_like(v, math.nan))
    return v.flatten(-2)


def _exact_tables(case, seed):
    d = _draw_tables(case, seed)
    P = case["page"]
    lens, new, table = d["lens"].tolist(), d["new"].tolist(), d["table"].tolist()
    free = d["free"].tolist()
    count = int(d["count"])
    after, cu, slot, pos = [], [0], [], []
    for r, n in enumerate(new):
        if n < 0:
            for j in range(-(-lens[r] // P)):
                free[count] = table[r][j]
                count += 1
    for r, n in enumerate(new):
        if n < 0:
            after.append(0)
            cu.append(cu[-1])
            continue
        for j in range(-(-lens[r] // P), -(-(lens[r] + n) // P)):
            count -= 1
            table[r][j] = free[count]
        for t in range(lens[r], lens[r] + n):
            slot.append(table[r][t // P] * P + t % P)
            pos.append(t)
        after.append(lens[r] + n)
        cu.append(cu[-1] + n)
    pad = case["slots"] - len(slot)
    i32 = dict(dtype=torch.int32, device=DEV)
    return (torch.tensor(after, **i32), torch.tensor(cu, **i32),
            torch.tensor(slot + [-1] * pad, dtype=torch.int64, device=DEV), torch.tensor(pos + [-1] * pad, **i32),
            torch.tensor([count], **i32), torch.tensor(table, **i32), torch.tensor(free, **i32))


def exact(case, seed):
    if case["op"] == "tables":
        return _exact_tables(case, seed)
    if case["op"] in ("store", "load"):
        k, v, _, _ = _draw_rows(case, seed)
        return tuple(torch.cat([_exact_values(c) for c in x.split(8192)]).to(torch.bfloat16) for x in (k, v))
    a = _draw_attn(case, seed)
    T, Hq, d = a["q"].shape
    Hkv = case["Hkv"]
    G = Hq // Hkv
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    for r, (L, n) in enumerate(zip(a["lens"], a["qlens"])):
        kb, qb = a["cu_k"][r], a["cu_q"][r]
        for h in range(Hkv):
            kk, vv = _exact_values(a["k"][kb:kb + L, h]), _exact_values(a["v"][kb:kb + L, h])
            for i0 in range(0, n, 256):
                i1 = min(n, i0 + 256)
                qq = a["q"][qb + i0:qb + i1, h * G:(h + 1) * G].double().reshape(-1, d)
                s = (qq @ kk.t()).reshape(i1 - i0, G, L) / math.sqrt(d)
                if case["causal"]:
                    i = torch.arange(i0, i1, device=DEV).view(-1, 1, 1)
                    s.masked_fill_(torch.arange(L, device=DEV) > L - n + i, -math.inf)
                z = torch.logsumexp(s, -1, keepdim=True)
                o[qb + i0:qb + i1, h * G:(h + 1) * G] = torch.exp(s - z) @ vv
                lse[h * G:(h + 1) * G, qb + i0:qb + i1] = z.squeeze(-1).t()
    return o, lse
