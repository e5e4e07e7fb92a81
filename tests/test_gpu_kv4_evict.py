"""Eviction by accumulated attention weight on the GPU: against plain loops (whole numbers, equal), the moves bit by
bit, and together with what a serving loop does around it."""

import math
import random

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import kv4 as O
from oracle import kv4_evict as E
from oracle import rope as OR

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra(lib_path):
    import context_ring_attention_step_gb300 as m
    m.load_library(lib_path)
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def draw(seed, lens, page, width=None, spare=5, kind="spread"):
    """Block table with pages in random order, sums of all slots, and the free pages."""
    rng = np.random.default_rng(seed)
    held = [max(0, -(-n // page)) for n in lens]
    width = width or max(held + [0]) + 2
    N = sum(held) + spare
    ids = rng.permutation(N)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    w = np.exp(2 * rng.standard_normal(N * page)).astype(np.float32)
    if kind == "ties":                                           # few values: the lowest indices decide
        w = rng.integers(0, 4, N * page).astype(np.float32)
    elif kind == "zeros":
        w[:] = 0
    elif kind == "odd":                                          # what is no positive number counts as 0
        w[rng.random(N * page) < 0.3] = np.nan
        w[rng.random(N * page) < 0.2] = -np.inf
        w[rng.random(N * page) < 0.1] = np.inf
        w[rng.random(N * page) < 0.1] = -1
        w[rng.random(N * page) < 0.1] = -0.0
        w[rng.random(N * page) < 0.1] = 1e-42                    # below the normal numbers
    free = np.full(N, -7, dtype=np.int32)
    free[:spare] = ids[at:]
    return table, w, free, spare, N


def run(ra, table, w, lens, budgets, page, moves, slack, recent, sinks, free=None, count=0, in_place=False, ws=None, pad=0):
    tb = torch.full((table.shape[0], table.shape[1] + pad), -9, dtype=torch.int32).cuda()[:, :table.shape[1]]
    tb.copy_(torch.tensor(table))
    ln, fr = i32(lens), None if free is None else i32(free)
    ct = None if free is None else i32([count])
    out = ra.kv4_evict_out(len(lens), moves)
    if in_place:
        out = out._replace(kv_lens=ln, free_count=ct if ct is not None else out.free_count)
    e = ra.kv4_evict(torch.tensor(w).cuda(), tb, ln, i32(budgets), page, moves, slack, recent, sinks, fr, ct, ws, out)
    assert np.array_equal(tb.cpu().numpy(), table)               # the block table stays
    return (e.kv_lens.tolist(), e.dropped.tolist(), e.src_slots.tolist(), e.dst_slots.tolist(), int(e.free_count),
            None if fr is None else fr.tolist()), int(e.status), e


def check(ra, table, w, lens, budgets, page, moves, slack, recent, sinks, free, count, status=0, **kw):
    *want, refused = E.evict(w, table.tolist(), lens, budgets, page, moves, slack, recent, sinks, free.tolist(), count)
    got, code, e = run(ra, table, w, lens, budgets, page, moves, slack, recent, sinks, free, count, **kw)
    assert got == tuple(want)
    assert code == status and bool(refused) == bool(status)
    return e


@pytest.mark.parametrize("kind", ["spread", "ties", "zeros", "odd"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("in_place", [False, True])
def test_small_batches(ra, kind, page, in_place):
    rng = random.Random(page)
    lens = [0, 1, 20, 31, 32, 33, 64, 100, 257, 1000, 1023, 7, 50, 2000, 129]
    for slack, recent, sinks in ((0, 0, 0), (0, 1, 0), (5, 3, 2), (16, 17, 4)):
        budgets = [rng.choice([0, 1, n // 2, max(0, n - 1), max(0, n - slack - 1), n, n + 3, -1]) for n in lens]
        budgets = [b if b < 0 else max(b, recent + sinks) for b in budgets]
        table, w, free, count, N = draw(page + slack, lens, page, kind=kind)
        check(ra, table, w, lens, budgets, page, 2000, slack, recent, sinks, free, count, in_place=in_place, pad=3)


@pytest.mark.parametrize("L,B,page", [(8193, 1000, 64), (40000, 4096, 128), (131072, 8192, 64), (131071, 131000, 16),
                                      (131072, 0, 256), (70001, 64, 32)])
@pytest.mark.parametrize("kind", ["spread", "ties", "zeros"])
def test_one_long_request(ra, L, B, page, kind):
    """A cluster of up to 16 CTAs; equal sums are told apart across them."""
    table, w, free, count, N = draw(L, [L], page, kind=kind)
    check(ra, table, w, [L], [B], page, max(1, min(B, L - B)), 0 if B == 0 else 40, 0 if B == 0 else 41, min(B, 4), free, count)


def test_more_tokens_than_shared_memory_holds(ra):
    """Keys beyond what a CTA keeps are made again from the sums."""
    L, B = 8 * 40960 + 30000, 5000
    table, w, free, count, N = draw(3, [L], 256)
    check(ra, table, w, [L], [B], 256, B, 10, 11, 3, free, count)
    lens = [50001] * 80                                          # (160 requests and more: one CTA each)
    lens += [11] * 90
    table, w, free, count, N = draw(4, lens, 256, kind="ties")
    check(ra, table, w, lens, [3000] * len(lens), 256, 3000, 0, 0, 1, free, count)


@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_more_tokens_than_a_cluster_holds(ra, kind):
    L, B = 16 * 40960 + 30000, 5000
    table, w, free, count, N = draw(5, [L], 256, kind=kind)
    check(ra, table, w, [L], [B], 256, B, 10, 11, 3, free, count)


@pytest.mark.parametrize("L,B", [(40, 20), (9000, 700)])
def test_sums_at_any_address(ra, L, B):
    """Sums begin at any multiple of four bytes."""
    table, w, free, count, N = draw(L, [L, 33], 16)
    want = E.evict(w, table.tolist(), [L, 33], [B, 16], 16, B, 0, 1, 2)
    for shift in (1, 2, 3):
        buf = torch.full((len(w) + 4,), float("nan")).cuda()
        buf[shift:shift + len(w)] = torch.tensor(w).cuda()
        e = ra.kv4_evict(buf[shift:shift + len(w)], torch.tensor(table).cuda(), i32([L, 33]), i32([B, 16]), 16, B, 0, 1, 2,
                         check=True)
        assert (e.kv_lens.tolist(), e.dropped.tolist(), e.src_slots.tolist(), e.dst_slots.tolist()) == tuple(want[:4])


@pytest.mark.parametrize("R", [127, 600, 4096])
def test_many_requests(ra, R):
    rng = random.Random(R)
    lens = [rng.randrange(0, 200) for _ in range(R)]
    budgets = [rng.choice([-1, 10, 50, 100]) for _ in range(R)]
    table, w, free, count, N = draw(R, lens, 16, kind="ties")
    check(ra, table, w, lens, budgets, 16, 100, 3, 4, 2, free, count)


def test_without_a_free_list(ra):
    table, w, _, _, _ = draw(5, [100, 30], 16)
    want = E.evict(w, table.tolist(), [100, 30], [40, 40], 16, 60, 0, 0, 0)
    got, code, _ = run(ra, table, w, [100, 30], [40, 40], 16, 60, 0, 0, 0)
    assert code == 0 and got[:4] == tuple(want[:4]) and got[4] == 0
    e = ra.kv4_evict(torch.tensor(w).cuda(), torch.tensor(table).cuda(), i32([100, 30]), i32([40, 40]), 16, 60,
                     free_count=i32([12]))
    assert int(e.free_count) == 12                               # the count is handed on


def test_requests_that_cannot_be_cut_are_left_alone(ra):
    lens, budgets = [300, 200, 100, 400], [100, 100, 50, 64]
    args = dict(page=16, moves=100, slack=4, recent=5, sinks=2)
    for change, status in (("page", 1001), ("far page", 1001), ("length", 1002), ("long", 1002), ("budget", 1007), ("moves", 1008)):
        table, w, free, count, N = draw(8, lens, 16)
        ln, bd, a = list(lens), list(budgets), dict(args)
        if change == "page":
            table[3, 9] = -1
        elif change == "far page":
            table[3, 24] = N
        elif change == "length":
            ln[1] = -4
        elif change == "long":
            ln[1] = table.shape[1] * 16 + 1
        elif change == "budget":
            bd[2] = 6
        else:
            a["moves"] = 40
        e = check(ra, table, w, ln, bd, a["page"], a["moves"], a["slack"], a["recent"], a["sinks"], free, count, status=status)
        with pytest.raises(ra.RingAttnError) as err:
            ra.kv4_status(e.status)
        assert err.value.status == (4 if status == 1008 else 1)


@pytest.mark.parametrize("count", [-1, 6, 1 << 30])
def test_pages_that_do_not_fit_the_free_list(ra, count):
    """Nothing is dropped, not even by the requests that could be."""
    lens = [300, 200, 10]
    table, w, free, _, N = draw(9, lens, 16)
    before = torch.tensor(free[:12].copy())
    for in_place in (False, True):
        got, code, _ = run(ra, table, w, lens, [100, 100, 100], 16, 100, 0, 0, 0, free[:12], count, in_place)
        assert code == 1006
        assert got[0] == lens and got[1] == [0, 0, 0] and got[4] == count and got[5] == before.tolist()
        assert got[2] == got[3] == [[-1] * 100] * 3


def test_two_calls_at_once_and_a_captured_one(ra):
    lens, page = [500, 4000, 77], 32
    table, w, free, count, N = draw(11, lens, page)
    want = run(ra, table, w, lens, [100, 1000, 60], page, 1000, 8, 9, 3, free, count)[0]
    torch.cuda.synchronize()
    wt, tb, ln, bd = torch.tensor(w).cuda(), torch.tensor(table).cuda(), i32(lens), i32([100, 1000, 60])
    fr, ct = [i32(free) for _ in range(3)], i32([count])
    got = []
    for s, f in zip([torch.cuda.Stream() for _ in range(2)], fr):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append((ra.kv4_evict(wt, tb, ln, bd, page, 1000, 8, 9, 3, f, ct), f))
    torch.cuda.synchronize()
    ws, out = ra.kv4_evict_workspace(3), ra.kv4_evict_out(3, 1000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.kv4_evict(wt, tb, ln, bd, page, 1000, 8, 9, 3, fr[2], ct, ws, out)
    for turn in range(3):
        graph.replay()
        torch.cuda.synchronize()
        if turn == 0:
            got.append((out, fr[2].clone()))
            ln[1] = 900                                          # lengths are read by the kernel
        else:
            assert out.kv_lens.tolist() == [100, 900, 60] and out.dropped.tolist() == [400, 0, 17]
            break
    e = got.pop()
    got = [(x.kv_lens.tolist(), x.dropped.tolist(), x.src_slots.tolist(), x.dst_slots.tolist(), int(x.free_count), f.tolist())
           for x, f in got]
    assert got[0] == want and got[1] == want
    assert e[1].tolist() == want[5]


@pytest.mark.parametrize("d,H,page", [(64, 3, 16), (128, 8, 64), (256, 2, 32)])
def test_moves_are_exact(ra, d, H, page):
    rng = np.random.default_rng(d)
    n, N = 700, 2000 // page + 1
    cache = ra.Kv4Cache(N, page, H, d)
    cache.pages.random_(0, 256, generator=torch.Generator("cuda").manual_seed(d))
    k, v = (torch.tensor(rng.standard_normal((2 * n, H, d)) * 3).to(torch.bfloat16).cuda() for _ in range(2))
    k[5, 0, 7] = float("nan")
    slots = torch.tensor(rng.permutation(N * page)[:2 * n]).cuda()
    ra.kv4_store(cache, k, v, slots)
    w = torch.rand(N * page).cuda()
    src, dst = slots[:n].clone(), slots[n:].clone()
    src[3], dst[4], src[9], dst[10] = -1, -5, N * page, 1 << 40   # left out
    every = torch.arange(N * page).cuda()
    k0, v0 = ra.kv4_load(cache, every)
    w0 = w.clone()
    ra.kv4_move(cache, src.view(7, 100), dst.view(7, 100), weights=w0)
    go = torch.ones(n, dtype=torch.bool)
    go[[3, 4, 9, 10]] = False
    k1, v1 = ra.kv4_load(cache, every)
    want_k, want_v, want_w = k0.clone(), v0.clone(), w.clone()
    want_k[dst[go]], want_v[dst[go]], want_w[dst[go]] = k0[src[go]], v0[src[go]], w[src[go]]
    for a, b in ((k1, want_k), (v1, want_v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))   # NaN and garbage too
    assert torch.equal(w0, want_w)
    with pytest.raises(ValueError, match="twice"):
        ra.kv4_move(cache, src[:2], dst[:1].expand(2).contiguous(), check=True)
    with pytest.raises(ValueError, match="occurs"):
        ra.kv4_move(cache, slots[:2], slots[1:3], check=True)
    ra.kv4_move(cache, src[:0], dst[:0])


def test_moves_beyond_32_bits(ra):
    page, d = 256, 64
    N = (1 << 32) // (256 // 16 * 18 * d) + 900
    cache = ra.Kv4Cache(N, page, 1, d)
    k = torch.randn(300, 1, d).to(torch.bfloat16).cuda()
    src = (torch.arange(300) + (N - 2) * page).cuda()
    dst = (torch.arange(300) + 5).cuda()
    ra.kv4_store(cache, k, -k, src)
    ra.kv4_move(cache, src, dst)
    a, b = ra.kv4_load(cache, src), ra.kv4_load(cache, dst)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and bool((b[0] != 0).any())
    ra.kv4_move(cache, dst, src + 300)                           # the cache ends after 212 of them
    last = ra.kv4_load(cache, src + 300)[0]
    assert torch.equal(last[:212], b[0][:212]) and not bool(last[212:].any())


def test_refusals(ra):
    table, w, free, count, N = draw(12, [100, 60], 16)
    wt, tb, ln, bd = torch.tensor(w).cuda(), torch.tensor(table).cuda(), i32([100, 60]), i32([50, 50])
    ok = dict(weights=wt, block_table=tb, kv_lens=ln, budgets=bd, page_size=16, max_moves=50)
    for kw, word in ((dict(weights=wt.double()), "weights"), (dict(weights=wt[:-1]), "multiple"), (dict(budgets=bd.long()), "budgets"),
                     (dict(budgets=bd[:1]), "budgets"), (dict(block_table=tb[:1]), "block_table"), (dict(kv_lens=ln.cpu()), "GPU"),
                     (dict(free_pages=i32(free)), "free_count"), (dict(out=ra.kv4_evict_out(2, 49)), "src_slots")):
        with pytest.raises(ValueError, match=word):
            ra.kv4_evict(**dict(ok, **kw))
    for kw, word in ((dict(page_size=48, weights=wt[:48]), "page_size"), (dict(max_moves=0), "max_moves"), (dict(slack=-1), "slack"),
                     (dict(recent=2), "recent"), (dict(sinks=-1), "sinks"),
                     (dict(workspace=torch.zeros(128, dtype=torch.uint8).cuda()), "workspace"),
                     (dict(out=ra.kv4_evict_out(2, 50)._replace(dropped=ln)), "lies over"),
                     (dict(out=ra.kv4_evict_out(2, 50)._replace(kv_lens=bd)), "lies over")):
        with pytest.raises(ra.RingAttnError, match=word):
            ra.kv4_evict(**dict(ok, **kw))
    with pytest.raises(ra.RingAttnError):
        ra.kv4_evict(wt, tb[:0], ln[:0], bd[:0], 16, 5)          # no requests
    cache = ra.Kv4Cache(N, 16, 2, 64)
    s = torch.zeros(4, dtype=torch.int64).cuda()
    for a, b, kw, word in ((s, s[:3], {}, "dst_slots"), (s.int(), s, {}, "src_slots"), (s, s, dict(weights=wt[:-1]), "weights")):
        with pytest.raises(ValueError, match=word):
            ra.kv4_move(cache, a, b, **kw)
    with pytest.raises(ra.RingAttnError, match="lies over"):
        ra.kv4_move(cache, cache.pages.view(-1)[:32].view(torch.int64), s)


# ------------------------------------------------------------------ all of it together

def test_prompt_tokens_and_evictions(ra):
    """A small model's attention: normed and rotated rows, a ring-attention prompt, then captured steps of single
    tokens whose requests are cut whenever they pass their budget.  Followed in float64 by the sets of cached tokens."""
    Hq, Hkv, d, page, B, slack, recent, sinks = 4, 2, 64, 16, 48, 8, 6, 2
    prompts, steps, scale = [40, 60], 30, 1 / math.sqrt(64)
    R, N, W = 2, 16, 8
    g = torch.Generator().manual_seed(77)
    total = sum(prompts) + R * steps
    raw = torch.randn(total, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    rotary, freq = ra.Rotary(d, base=100.0), OR.frequencies(d, 100.0)
    cache = ra.Kv4Cache(N, page, Hkv, d)
    table, free, count = torch.full((R, W), -1, dtype=torch.int32).cuda(), i32(list(range(N))), i32([N])
    weights = torch.zeros(N * page).cuda()
    budgets, gone = i32([B] * R), torch.zeros(R, dtype=torch.int32).cuda()
    lens = i32([0, 0])

    # ---- the prompts: norm and rotation, ring attention, cache, and their tokens' weights
    T = sum(prompts)
    qkv = raw[:T].cuda()
    cu = [0, prompts[0], T]
    q, k = ra.qk_norm_rope_fwd(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], ra.rope_positions(cu), rotary, wq, wk)
    v = qkv[:, Hq + Hkv:].contiguous()
    o, lse = ra.ring_attn_fwd(q, k, v, cu, 2, scale=scale, check=True)
    ro, rl = A.attention_fwd(q.cpu(), k.cpu(), v.cpu(), cu, True, scale)
    assert np.abs(f64(o) - ro).max() < 2e-2 and np.abs(f64(lse) - rl).max() < 1e-3
    new = i32(prompts)
    step = ra.kv4_tables(lens, new, table, page, T, free, count, check=True)
    ra.kv4_store(cache, k, v, step.slot_map, check=True)
    o, lse = ra.kv4_attention(q, cache, table, step.kv_lens, step.cu_new, scale=scale, max_q_len=60, check=True)
    ra.kv4_weights(q, cache, table, step.kv_lens, step.cu_new, lse, weights, new_lens=new, scale=scale, max_q_len=60, check=True)

    # ---- the same in float64: cached rows and their sums, by request, in order of the cache's places
    kr, vr = (f64(x) for x in ra.kv4_load(cache, step.slot_map))
    keys, vals = [kr[:40], kr[40:]], [vr[:40], vr[40:]]
    sums = E.weights(f64(q), keys, prompts, cu, f64(lse), True, scale)
    held = table.tolist()

    def slots_of(r, n):
        return [held[r][i // page] * page + i % page for i in range(n)]

    def agree():
        for r in range(R):
            n = len(keys[r])
            s = torch.tensor(slots_of(r, n)).cuda()
            gk, gv = ra.kv4_load(cache, s)
            assert np.array_equal(f64(gk), keys[r]) and np.array_equal(f64(gv), vals[r])
            assert np.allclose(f64(weights[s]), sums[r], rtol=1e-4, atol=1e-6)

    lens, count = step.kv_lens, step.free_count
    agree()

    # ---- a captured step: rotation at the true positions, tables, store, attention, weights, eviction, moves
    rows = torch.zeros(R, Hq + 2 * Hkv, d, dtype=torch.bfloat16).cuda()
    ones, out = i32([1] * R), ra.kv4_tables_out(R, R)._replace(kv_lens=lens, free_count=count)
    eo = ra.kv4_evict_out(R, slack + 1)._replace(kv_lens=lens, free_count=count)
    aw, ew = ra.kv4_attention_workspace(cache, R, Hq, 1), ra.kv4_evict_workspace(R)
    qo, ko = torch.empty(R, Hq, d, dtype=torch.bfloat16).cuda(), torch.empty(R, Hkv, d, dtype=torch.bfloat16).cuda()
    res = (torch.empty(R, Hq, d).cuda(), torch.empty(Hq, R).cuda())

    def one_step():
        s = ra.kv4_tables(lens, ones, table, page, R, free, count, out=out)
        ra.qk_norm_rope_fwd(rows[:, :Hq], rows[:, Hq:Hq + Hkv], s.positions + gone, rotary, wq, wk, out=(qo, ko))
        ra.kv4_store(cache, ko, rows[:, Hq + Hkv:], s.slot_map)
        ra.kv4_attention(qo, cache, table, lens, s.cu_new, scale=scale, max_q_len=1, workspace=aw, out=res, o_fp32=True)
        ra.kv4_weights(qo, cache, table, lens, s.cu_new, res[1], weights, new_lens=ones, scale=scale, max_q_len=1, workspace=aw)
        e = ra.kv4_evict(weights, table, lens, budgets, page, slack + 1, slack, recent, sinks, free, count, ew, eo)
        ra.kv4_move(cache, e.src_slots, e.dst_slots, weights=weights)
        gone.add_(e.dropped)

    graph = torch.cuda.CUDAGraph()
    state = [x.clone() for x in (table, free, count, lens, weights, gone, cache.pages)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one_step()                                               # (first calls outside the capture)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((table, free, count, lens, weights, gone, cache.pages), state):
        x.copy_(y)
    with torch.cuda.graph(graph):
        one_step()
    seen, cuts = list(prompts), 0
    for i in range(steps):
        new_rows = raw[T + R * i:T + R * (i + 1)]
        rows.copy_(new_rows)
        before = [len(x) for x in keys]
        graph.replay()
        torch.cuda.synchronize()
        ra.kv4_status(out.status)
        ra.kv4_status(aw)
        ra.kv4_status(eo.status)
        held = table.tolist()
        # rotation at the number of tokens seen so far
        want = OR.forward(f64(new_rows[:, :Hq]), seen, freq, False, f64(wq), 1e-6)
        assert np.abs(f64(qo) - want).max() < 2.0 ** -8 * np.abs(want).max() * 1.1
        kn, vn = O.rounded(f64(ko)), O.rounded(f64(new_rows[:, Hq + Hkv:]))
        for r in range(R):
            keys[r], vals[r] = np.concatenate([keys[r], kn[r:r + 1]]), np.concatenate([vals[r], vn[r:r + 1]])
            sums[r] = np.concatenate([sums[r], [0.0]])
            seen[r] += 1
        o64, l64 = O.attention(f64(qo), keys, vals, [n + 1 for n in before], [0, 1, 2], True, scale)
        assert np.abs(f64(res[0]) - o64).max() < 5e-3 and np.abs(f64(res[1]) - l64).max() < 1e-3
        add = E.weights(f64(qo), keys, [n + 1 for n in before], [0, 1, 2], f64(res[1]), True, scale)
        for r in range(R):
            sums[r] = sums[r] + add[r]
            if before[r] + 1 > B + slack:
                # the GPU's own choice, which close sums may decide otherwise than float64: checked by what it implies
                s, t = (x[r].tolist() for x in (eo.src_slots, eo.dst_slots))
                where = {x: j for j, x in enumerate(slots_of(r, before[r] + 1))}
                pairs = [(where[a], where[b]) for a, b in zip(s, t) if a >= 0]
                drop = [b for _, b in pairs] + [j for j in range(B, before[r] + 1) if j not in {a for a, _ in pairs}]
                assert len(drop) == before[r] + 1 - B and not set(drop) & (set(range(sinks)) | set(range(before[r] + 1 - recent, before[r] + 1)))
                rest = [j for j in range(sinks, before[r] + 1 - recent) if j not in drop]
                assert max(sums[r][drop]) <= min(sums[r][rest]) * (1 + 1e-4)
                for a, b in pairs:
                    assert a >= B > b
                    keys[r][b], vals[r][b], sums[r][b] = keys[r][a], vals[r][a], sums[r][a]
                keys[r], vals[r], sums[r] = keys[r][:B], vals[r][:B], sums[r][:B]
                cuts += 1
        assert lens.tolist() == [len(x) for x in keys]
        assert gone.tolist() == [s - len(x) for s, x in zip(seen, keys)]
        agree()
    assert cuts >= 4
    # every page is in the free list or the block table, once
    used = [held[r][j] for r in range(R) for j in range(-(-len(keys[r]) // page))]
    assert sorted(used + free.tolist()[:int(count)]) == list(range(N))
