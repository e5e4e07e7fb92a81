"""4-bit key/value cache on the GPU against the fp64 oracle.

Store, load and the tables are exact.  Attention's tolerance, derived for
every case from its inputs (see ``bounds``):
  * S is accumulated in fp32 from exact products: D terms, each sum off by at
    most one unit in the last place (tensor cores may truncate: 2^-23) of the
    sum of magnitudes; that is an absolute error e_s of the exponent, and a
    relative one of every p (twice with the normaliser);
  * p goes into P.V as fp16: 2^-11 relative at the most coarse reading of half a
    step (finfo(fp16).eps / 2 = 2^-11), and 2^-25 / 2^6 absolute;
  * 2^x and log2 approximations and the merge weights: 2^-20;
  * O and l add at most L terms in fp32, 16 at a time in the products;
  * bf16 outputs round by half a step: finfo(bf16).eps / 2 relative.
"""

import math
import random

import numpy as np
import pytest
import torch

from oracle import kv4 as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra(lib_path):
    import context_ring_attention_step_gb300 as m
    m.load_library(lib_path)
    return m


def bf16(rng, *shape, scale=1.0):
    return torch.tensor(rng.standard_normal(shape) * scale, dtype=torch.float32).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ store and load

def hard_rows(rng, T, H, d):
    """Rows with ties of both formats, tiny, huge, zero and non-finite groups."""
    x = rng.standard_normal((T, H, d)) * np.exp2(rng.integers(-24, 20, (T, H, 1)))
    g = x.reshape(T, H, d // 16, 16)
    kind = rng.integers(0, 12, (T, H, d // 16))
    ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
    for i, e in enumerate((-12, 0, 9)):
        g[kind == i] = ties * 2.0 ** e                           # elements on the borders
    g[kind == 4] = rng.integers(-255, 256, g[kind == 4].shape)   # amax / 6 on and off the scales' borders
    g[kind == 5] = 0
    g[kind == 6] *= 1e30
    g[kind == 7] = rng.choice([0, 2.0 ** -17, 2.0 ** -18 * 3, -2.0 ** -20, 2.0 ** -15], g[kind == 7].shape)
    g[kind == 8, 3] = np.inf
    g[kind == 9, 15] = np.nan
    return torch.tensor(x).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,page,T", [(1, 16, 1), (3, 32, 77), (8, 64, 333), (2, 256, 600)])
def test_store_load_are_exact(ra, d, H, page, T):
    rng = np.random.default_rng(100 * d + T)
    pages = T // page + 3
    k, v = hard_rows(rng, T, H, d), hard_rows(rng, T, H, d)
    slots = torch.tensor(rng.permutation(pages * page)[:T])
    skip = torch.tensor(rng.random(T) < 0.1)
    given = torch.where(skip, torch.tensor(rng.choice([-1, -7, pages * page, 1 << 40], T)), slots)
    cache = ra.Kv4Cache(pages, page, H, d)
    # rows of a fused projection: q, k, v of a token one after the other
    qkv = torch.cat([k, torch.zeros(T, 2, d, dtype=torch.bfloat16), v], dim=1).cuda()
    ra.kv4_store(cache, qkv[:, :H], qkv[:, H + 2:], given.cuda(), check=False)
    ko, vo = ra.kv4_load(cache, slots.cuda())
    keep = (~skip).numpy()
    for got, x in ((ko, k), (vo, v)):
        want = O.rounded(f64(x))
        want[~keep] = 0                                          # never written: the fresh cache's zeros
        np.testing.assert_array_equal(f64(got), want)
    # skipped rows of a load are zero, repeated ones repeat
    again = torch.cat([slots[:5], slots[:5], torch.tensor([-1, pages * page, 1 << 62])]).cuda()
    k2, _ = ra.kv4_load(cache, again)
    n = min(5, T)
    assert torch.equal(torch.nan_to_num(k2[:n]), torch.nan_to_num(k2[n:2 * n])) and k2[2 * n:].eq(0).all()


@pytest.mark.parametrize("d,T", [(64, 39001), (128, 19458), (256, 9733)])
def test_store_load_of_a_long_prompt(ra, d, T):
    """Enough rows for the kernels that take four at a time: neighbouring slots, at every alignment, and gaps."""
    rng = np.random.default_rng(T)
    H, page = 8, 64
    pages = T // page + 4
    t = np.arange(T) + 3                                         # the first slot is not a multiple of four
    slots = rng.permutation(pages)[t // page] * page + t % page
    for a in rng.integers(0, T - 300, 40):                       # stretches that start at other alignments
        n = int(rng.integers(1, 200))
        slots[a:a + n] = np.roll(slots[a:a + n], int(rng.integers(1, 9)))
    given = slots.copy()
    given[rng.random(T) < 0.01] = -1
    given[rng.random(T) < 0.01] = pages * page + 5
    keep = (given >= 0) & (given < pages * page)
    k, v = bf16(rng, T, H, d), bf16(rng, T, H, d)
    cache = ra.Kv4Cache(pages, page, H, d)
    ra.kv4_store(cache, k.cuda(), v.cuda(), torch.tensor(given).cuda())
    ko, vo = ra.kv4_load(cache, torch.tensor(slots).cuda())
    kg, vg = ra.kv4_load(cache, torch.tensor(given).cuda())
    for got, again, x in ((ko, kg, k), (vo, vg, v)):
        want = O.rounded(f64(x))
        want[~keep] = 0
        np.testing.assert_array_equal(f64(got), want)
        assert torch.equal(got, again)
    some = torch.tensor(slots[5:5000:7]).cuda()                  # the same rows, one at a time
    assert torch.equal(ra.kv4_load(cache, some)[1], vo[5:5000:7])


@pytest.mark.parametrize("H,d", [(4096, 256), (4096, 64), (37, 128)])
def test_store_load_of_many_heads(ra, H, d):
    """Rows of more columns than a block has threads."""
    rng = np.random.default_rng(H + d)
    cache = ra.Kv4Cache(2, 16, H, d)
    k, v = bf16(rng, 5, H, d), bf16(rng, 5, H, d)
    slots = torch.tensor([20, 21, 22, 23, 3]).cuda()
    ra.kv4_store(cache, k.cuda(), v.cuda(), slots)
    for got, x in zip(ra.kv4_load(cache, slots), (k, v)):
        np.testing.assert_array_equal(f64(got), O.rounded(f64(x)))


def test_store_leaves_other_slots(ra):
    rng = np.random.default_rng(5)
    cache = ra.Kv4Cache(3, 32, 2, 128)
    cache.pages.random_(0, 256, generator=torch.Generator("cuda").manual_seed(1))
    others = torch.tensor([s for s in range(96) if s not in (17, 40)]).cuda()
    before = [t.clone() for t in ra.kv4_load(cache, others)]
    x = bf16(rng, 2, 2, 128).cuda()
    ra.kv4_store(cache, x, x, torch.tensor([17, 40]).cuda())
    for a, b in zip(before, ra.kv4_load(cache, others)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    np.testing.assert_array_equal(f64(ra.kv4_load(cache, torch.tensor([17, 40]).cuda())[0]), O.rounded(f64(x)))


def test_store_checks_slots(ra):
    cache = ra.Kv4Cache(2, 16, 1, 64)
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16).cuda()
    with pytest.raises(ValueError, match="twice"):
        ra.kv4_store(cache, x, x, torch.tensor([3, 3]).cuda(), check=True)
    with pytest.raises(ValueError, match="outside"):
        ra.kv4_store(cache, x, x, torch.tensor([3, 32]).cuda(), check=True)
    ra.kv4_store(cache, x, x, torch.tensor([-1, -1]).cuda(), check=True)
    ra.kv4_store(cache, x[:0], x[:0], torch.zeros(0, dtype=torch.int64).cuda(), check=True)


# ------------------------------------------------------------------ tables

def draw_tables(rng, R, page, width, alloc=True):
    lens = [rng.choice([0, rng.randrange(0, width * page + 1), rng.randrange(0, page + 1)]) for _ in range(R)]
    new = [rng.choice([-1, 0, 1, 1, 1, rng.randrange(0, 200)]) for _ in range(R)]
    new = [min(a, width * page - n) for n, a in zip(lens, new)]
    held = [-(-n // page) for n in lens]
    need = [-(-(n + max(a, 0)) // page) for n, a in zip(lens, new)]
    ids = list(range(sum(need) + sum(held) + 5))
    rng.shuffle(ids)
    table, at = [], 0
    for h, n in zip(held, need):
        m = h if alloc else n
        table.append(ids[at:at + m] + [-9] * (width - m))
        at += m
    free = ids[at:]
    pad = [-5] * (sum(held) + 3)
    return lens, new, table, free + pad, len(free)


def run_tables(ra, lens, new, table, page, slots, free=None, count=0, in_place=False, stride=None):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    tb = i32(table)
    if stride:
        wide = torch.full((len(table), stride), -77, dtype=torch.int32).cuda()
        wide[:, :tb.shape[1]] = tb
        tb = wide[:, :tb.shape[1]]
    fr = None if free is None else i32(free)
    ct = None if free is None else i32([count])
    ln = i32(lens)
    out = ra.kv4_tables_out(len(lens), slots)
    if in_place:
        out = out._replace(kv_lens=ln, free_count=ct if ct is not None else out.free_count)
    step = ra.kv4_tables(ln, i32(new), tb, page, slots, fr, ct, out=out)
    code = int(step.status)
    return (code, step.kv_lens.tolist(), step.cu_new.tolist(), step.slot_map.tolist(), step.positions.tolist(),
            None if ct is None else int(step.free_count), tb.tolist(), None if fr is None else fr.tolist())


@pytest.mark.parametrize("R,page,width", [(1, 16, 4), (3, 64, 9), (64, 64, 40), (200, 16, 30), (1025, 32, 12), (4096, 128, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_match_the_lists(ra, R, page, width, in_place):
    rng = random.Random(R + in_place)
    for spare in (0, 1, 137):
        lens, new, table, free, count = draw_tables(rng, R, page, width)
        slots = sum(max(a, 0) for a in new) + spare
        want = O.tables(lens, new, table, page, slots, free, count)
        got = run_tables(ra, lens, new, table, page, slots, free, count, in_place, stride=width + 3 if spare else None)
        assert got == (0,) + want


@pytest.mark.parametrize("R", [7, 1500])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_of_long_prompts(ra, R, in_place):
    """Many CTAs: prompts of thousands of tokens beside single tokens and requests that leave."""
    rng = random.Random(R)
    page, width = 32, 700
    lens = [rng.choice([0, 5, rng.randrange(0, 2000)]) for _ in range(R)]
    new = [rng.choice([-1, 1, 1, 1, 0]) for _ in range(R)]
    for r in rng.sample(range(R), 5):
        new[r] = rng.randrange(3000, 20000)
    held = [-(-n // page) for n in lens]
    total = sum(held) + sum(-(-(n + max(a, 0)) // page) for n, a in zip(lens, new))
    ids = list(range(total))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-3] * (width - h))
        at += h
    free = ids[at:] + [-5] * at
    slots = sum(max(a, 0) for a in new) + 1003
    want = O.tables(lens, new, table, page, slots, free, total - at)
    assert run_tables(ra, lens, new, table, page, slots, free, total - at, in_place) == (0,) + want


@pytest.mark.parametrize("R", [1, 33, 300])
def test_tables_map_only(ra, R):
    rng = random.Random(R)
    lens, new, table, _, _ = draw_tables(rng, R, 32, 20, alloc=False)
    slots = sum(max(a, 0) for a in new) + 9
    want = O.tables(lens, new, table, 32, slots)
    got = run_tables(ra, lens, new, table, 32, slots)
    assert got[:5] == (0,) + want[:4] and got[6] == table
    lens, new = [0] * 2, [40, 40]
    got = run_tables(ra, lens, new, [[3, -1], [7, 8]], 32, 80)
    assert got[3] == list(range(96, 128)) + [-1] * 8 + list(range(224, 264))


@pytest.mark.parametrize("change,code", [
    (dict(slots=99), 1004), (dict(count=1), 1005), (dict(count=-1), 1006), (dict(count=12), 1006),
    (dict(lens=[10, -1, 70]), 1002), (dict(lens=[10, 0, 129]), 1002), (dict(new=[30, -2, 3]), 1002),
    (dict(new=[119, -1, 3]), 1002), (dict(new=[2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]), 1002)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_refuse_whole_steps(ra, change, code, in_place):
    a = dict(lens=[10, 20, 70], new=[97, -1, 3], table=[[0, 1, 2, 3, 4, 5, 6, 7]] * 3, slots=100, count=8)
    a["free"] = list(range(10, 20))
    a.update(change)
    got = run_tables(ra, a["lens"], a["new"], a["table"], 16, a["slots"], a["free"], a["count"], in_place)
    assert got[0] == code
    assert got[1] == a["lens"] and got[2] == [0] * 4 and got[3] == [-1] * a["slots"] == got[4]
    assert got[5] == a["count"] and got[6] == a["table"] and got[7] == a["free"]
    step = ra.Kv4Tables(None, None, None, None, None, torch.tensor([code], dtype=torch.int32).cuda())
    with pytest.raises(ra.RingAttnError) as e:
        ra.kv4_status(step.status)
    assert e.value.status == (4 if code == 1005 else 1)


# ------------------------------------------------------------------ attention

class Case:
    """A cache with random pages, holding the keys and values of several requests."""

    def __init__(self, ra, seed, lens, qlens, Hq, Hkv, d, page, kscale=1.0, vscale=1.0, garbage=True, keys=None, values=None):
        rng = np.random.default_rng(seed)
        self.lens, self.qlens, self.Hq, self.Hkv, self.d = lens, qlens, Hq, Hkv, d
        held = [-(-n // page) for n in lens]
        N = sum(held) + 2
        ids = rng.permutation(N)
        width = max(held + [0]) + 2
        table = np.full((len(lens), width), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(held):
            table[r, :n] = ids[at:at + n]
            at += n
        self.cache = ra.Kv4Cache(N, page, Hkv, d)
        if garbage:   # what unused places hold must not matter: all bytes, NaN scales among them
            self.cache.pages.random_(0, 256, generator=torch.Generator("cuda").manual_seed(seed))
        self.keys, self.values = [], []
        for r, n in enumerate(lens):
            k = bf16(rng, n, Hkv, d, scale=kscale) if keys is None else keys[r]
            v = bf16(rng, n, Hkv, d, scale=vscale) if values is None else values[r]
            t = np.arange(n)
            slots = table[r, t // page].astype(np.int64) * page + t % page
            ra.kv4_store(self.cache, k.cuda(), v.cuda(), torch.tensor(slots).cuda())
            self.keys.append(O.rounded(f64(k)))
            self.values.append(O.rounded(f64(v)))
        self.cu = np.concatenate([[0], np.cumsum(qlens)]).astype(int).tolist()
        self.q = bf16(rng, self.cu[-1], Hq, d)
        self.table = torch.tensor(table).cuda()
        self.lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
        self.cu_t = torch.tensor(self.cu, dtype=torch.int32).cuda()

    def bounds(self, scale, o_fp32, want):
        """Absolute tolerances of o (array) and lse, as the module's docstring derives them."""
        L = max(self.lens + [1])
        qm = np.abs(f64(self.q)).max() if self.q.numel() else 0.0
        ks = max([np.nan_to_num(np.abs(k)).sum(-1).max() for k in self.keys if k.size] + [0.0])
        vm = max([np.nan_to_num(np.abs(v)).max() for v in self.values if v.size] + [0.0])
        e_s = scale * self.d * 2.0 ** -23 * qm * ks
        e = 2 * e_s + 2.0 ** -11 + 2.0 ** -20 + L * 2.0 ** -23
        tol_o = e * vm + L * 2.0 ** -31 * vm
        if not o_fp32:
            tol_o = tol_o + np.nan_to_num(np.abs(want)) * 2.0 ** -8
        return tol_o, e_s + 2.0 ** -20 + L * 2.0 ** -23 + 2.0 ** -22 * 20

    def check(self, ra, causal=True, scale=None, o_fp32=True, max_q_len=None, q=None):
        sc = scale or 1 / math.sqrt(self.d)
        want, wl = O.attention(f64(self.q), self.keys, self.values, self.lens, self.cu, causal, sc)
        o, lse = ra.kv4_attention((self.q.cuda() if q is None else q), self.cache, self.table, self.lens_t, self.cu_t,
                                  causal=causal, scale=scale, o_fp32=o_fp32, max_q_len=max_q_len, check=True)
        self.compare(f64(o), f64(lse), want, wl, sc, o_fp32)
        return o, lse

    def compare(self, o, lse, want, wl, sc, o_fp32):
        tol_o, tol_l = self.bounds(sc, o_fp32, want)
        assert np.array_equal(np.isnan(o), np.isnan(want))
        assert np.all(np.nan_to_num(np.abs(o - want)) <= tol_o), np.nanmax(np.abs(o - want) - tol_o)
        assert np.array_equal(np.isneginf(lse), np.isneginf(wl)) and np.array_equal(np.isnan(lse), np.isnan(wl))
        f = np.isfinite(wl)
        assert np.all(np.abs(lse[f] - wl[f]) <= tol_l), np.abs(lse[f] - wl[f]).max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 5, 8, 16])
@pytest.mark.parametrize("page", [16, 64])
def test_decode(ra, d, G, page):
    lens = [1, 2, 15, 16, 17, 31, 63, 64, 65, 0, 130, 1000]
    c = Case(ra, 7 * d + G, lens, [1] * len(lens), 2 * G, 2, d, page)
    c.check(ra, max_q_len=1)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 8, 2), (128, 7, 1), (256, 6, 2)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("qlens", [[2, 3, 1, 4, 0, 5, 8], [17, 0, 64, 1, 33, 5, 9]])
def test_several_tokens(ra, d, Hq, Hkv, causal, qlens):
    lens = [2, 40, 64, 100, 50, 333, 5]          # the last request brings more rows than it has keys
    c = Case(ra, 11 + d + sum(qlens), lens, qlens, Hq, Hkv, d, 32)
    c.check(ra, causal=causal, max_q_len=max(qlens))
    c.check(ra, causal=causal, o_fp32=False)     # max_q_len: the number of rows
    c.check(ra, causal=causal, max_q_len=1)      # a wrong bound costs time only
    c.check(ra, causal=causal, scale=0.3)


@pytest.mark.parametrize("d,Hq,Hkv,L", [(128, 4, 1, 4001), (64, 1, 1, 6000), (256, 2, 2, 2500), (128, 1, 1, 4096)])
def test_one_long_request_is_split(ra, d, Hq, Hkv, L):
    c = Case(ra, L, [L], [1], Hq, Hkv, d, 64)
    c.check(ra, max_q_len=1)


def test_prompt_part(ra):
    c = Case(ra, 3, [700, 512], [300, 257], 4, 2, 128, 64)
    c.check(ra, max_q_len=300)
    c.check(ra, causal=False, o_fp32=False, max_q_len=300)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 2), (128, 8, 1), (128, 3, 3), (256, 4, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_parts_among_single_tokens(ra, d, Hq, Hkv, causal):
    """Both kernels in one call: parts of prompts (one without a prefix), single tokens, and requests without rows."""
    lens = [700, 1, 0, 131, 129, 513, 260, 90]
    qlens = [1, 1, 0, 131, 65, 0, 200, 1]
    c = Case(ra, 17 + d, lens, qlens, Hq, Hkv, d, 64)
    c.check(ra, causal=causal, max_q_len=200)
    c.check(ra, causal=causal, max_q_len=200, o_fp32=False, scale=0.2)


@pytest.mark.parametrize("d,G,n,L", [(64, 2, 33, 3001), (64, 2, 70, 3001), (128, 4, 16, 5000), (128, 4, 30, 5000),
                                         (128, 1, 110, 2100), (128, 8, 129, 1111), (256, 4, 31, 2500), (256, 2, 90, 600)])
def test_one_prompt_part_is_split(ra, d, G, n, L):
    c = Case(ra, n + L, [L], [n], G, 1, d, 32)
    c.check(ra, max_q_len=n)
    first = ra.kv4_attention(c.q.cuda(), c.cache, c.table, c.lens_t, c.cu_t, max_q_len=n)
    again = ra.kv4_attention(c.q.cuda(), c.cache, c.table, c.lens_t, c.cu_t, max_q_len=n)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_more_rows_than_keys(ra):
    c = Case(ra, 19, [30, 0, 5], [100, 70, 80], 2, 1, 128, 16)
    o, lse = c.check(ra, max_q_len=100)
    assert o[:70].eq(0).all() and torch.isneginf(lse[:, :70]).all()


def test_uneven_scores_in_row_tiles(ra):
    rng = np.random.default_rng(13)
    L, d, n = 900, 128, 70
    ramp = np.concatenate([np.linspace(0.01, 30, 450), np.linspace(30, 0.01, 450)])
    k = torch.tensor(rng.standard_normal((L, 1, d)) * ramp[:, None, None]).to(torch.bfloat16)
    c = Case(ra, 13, [L], [n], 2, 1, d, 16, keys=[k])
    c.q[5] = 0
    c.q[6] *= 2.0 ** -100
    c.check(ra, max_q_len=n)


def test_uneven_scores_move_the_reference(ra):
    """Scores that grow along the keys by far more than the reference's headroom, and shrink again."""
    rng = np.random.default_rng(9)
    L, d = 900, 128
    ramp = np.concatenate([np.linspace(0.01, 30, 450), np.linspace(30, 0.01, 450)])
    k = torch.tensor(rng.standard_normal((1, 1, d)) * ramp[:, None, None]).to(torch.bfloat16)
    c = Case(ra, 9, [L], [3], 2, 1, d, 16, keys=[k])
    c.check(ra, max_q_len=3)


def test_wide_ranges_of_q(ra):
    rng = np.random.default_rng(10)
    c = Case(ra, 10, [200], [8], 2, 1, 128, 16)
    c.q = torch.tensor(rng.standard_normal((8, 2, 128)) * np.exp2([[-120], [-20], [-3], [0], [2], [3], [4], [5]])[:, :, None]).to(torch.bfloat16)
    c.q[0, 1] = 0
    c.check(ra, max_q_len=8)


def test_nan_stays_in_its_rows(ra):
    """A NaN value or key of a late token reaches the rows that see it, and no other."""
    rng = np.random.default_rng(12)
    for d, Hq, n in ((64, 2, 40), (128, 4, 20), (256, 2, 40), (64, 3, 40), (128, 4, 40), (256, 3, 40)):
        L = 150                                                  # both kernels: fewer than 96 rows, and more
        k, v = bf16(rng, L, 1, d), bf16(rng, L, 1, d)
        v[140, 0, 3] = float("nan")
        v[141, 0, d - 1] = float("inf")
        c = Case(ra, d, [L], [n], Hq, 1, d, 16, keys=[k], values=[v])
        c.check(ra, max_q_len=n)
        assert not np.isnan(f64(c.check(ra, max_q_len=n)[0])[:n - 10]).any()
        k[149, 0, 5] = float("nan")
        c = Case(ra, d, [L], [n], Hq, 1, d, 16, keys=[k], values=[v])
        c.check(ra, max_q_len=n)
        c.check(ra, max_q_len=1)


def test_strided_q_and_rows_behind_the_last(ra):
    c = Case(ra, 21, [40, 90], [1, 2], 4, 2, 64, 16)
    T = 6                                                        # three rows more than the requests bring
    fused = torch.full((T, 8, 64), float("nan"), dtype=torch.bfloat16).cuda()
    fused[:3, :4] = c.q.cuda()
    o = torch.full((T, 4, 64), 7.0, device="cuda")
    lse = torch.full((4, T), 5.0, device="cuda")
    ra.kv4_attention(fused[:, :4], c.cache, c.table, c.lens_t, c.cu_t, o_fp32=True, max_q_len=2, out=(o, lse), check=True)
    want, wl = O.attention(f64(c.q), c.keys, c.values, c.lens, c.cu, True, 1 / 8)
    c.compare(f64(o[:3]), f64(lse[:, :3]), want, wl, 1 / 8, True)
    assert o[3:].eq(7).all() and lse[:, 3:].eq(5).all()


@pytest.mark.parametrize("longest", [1, 64])                     # 64: single tokens beside the row-tile kernel
def test_refused_contents_are_reported_and_stay_in_bounds(ra, longest):
    c = Case(ra, 31, [40, 90, 33], [1, 1, 1], 4, 2, 64, 16)
    q = c.q.cuda()
    good = ra.kv4_attention(q, c.cache, c.table, c.lens_t, c.cu_t, max_q_len=longest, check=True)[0]

    def refused(match, table=c.table, lens=c.lens_t, cu=c.cu_t):
        ws = ra.kv4_attention_workspace(c.cache, 3, 4, longest)
        o, _ = ra.kv4_attention(q, c.cache, table, lens, cu, max_q_len=longest, workspace=ws)
        with pytest.raises(ra.RingAttnError, match=match):
            ra.kv4_status(ws)
        ra.kv4_attention(q, c.cache, c.table, c.lens_t, c.cu_t, max_q_len=longest, workspace=ws, check=True)  # fresh status
        return o
    for bad in (-1, c.cache.num_pages, 2 ** 31 - 1, -2 ** 31):
        t = c.table.clone()
        t[1, 2] = bad
        o = refused("page", table=t)
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2]) and torch.isfinite(o).all()
    for bad in (-1, c.table.shape[1] * 16 + 1, 2 ** 31 - 1):
        x = c.lens_t.clone()
        x[1] = bad
        refused("length|page", lens=x)
    x = c.lens_t.clone()
    x[1] = -5
    o = refused("length", lens=x)
    assert torch.equal(o[0], good[0]) and o[1].eq(0).all() and torch.equal(o[2], good[2])
    for cu in ([0, 1, 2, 4], [0, 2, 1, 3], [-1, 1, 2, 3], [0, 1, 2, 2 ** 31 - 1]):
        refused("offsets", cu=torch.tensor(cu, dtype=torch.int32).cuda())


def test_bad_pages_in_row_tiles(ra):
    """A key on a page outside the cache is left out of every row, the others stay."""
    c = Case(ra, 33, [300, 200], [70, 80], 2, 1, 128, 16)
    ws = ra.kv4_attention_workspace(c.cache, 150, 2, 80)
    for bad in (-1, c.cache.num_pages, 2 ** 31 - 1, -2 ** 31):
        t = c.table.clone()
        t[0, 3] = bad
        o, lse = ra.kv4_attention(c.q.cuda(), c.cache, t, c.lens_t, c.cu_t, o_fp32=True, max_q_len=80, workspace=ws)
        with pytest.raises(ra.RingAttnError, match="page"):
            ra.kv4_status(ws)
        keys, values = [np.delete(x[0], np.s_[48:64], axis=0) for x in (c.keys, c.values)]
        want, wl = O.attention(f64(c.q), [keys, c.keys[1]], [values, c.values[1]], [284, 200], c.cu, True, 1 / math.sqrt(128))
        c.compare(f64(o), f64(lse), want, wl, 1 / math.sqrt(128), True)


def test_empty_calls(ra):
    c = Case(ra, 41, [0, 0], [1, 2], 4, 2, 64, 16)
    o, lse = c.check(ra, max_q_len=2)
    assert o.eq(0).all() and torch.isneginf(lse).all()
    e = torch.zeros(0, 4, 64, dtype=torch.bfloat16).cuda()
    z = torch.zeros(3, dtype=torch.int32).cuda()
    o, lse = ra.kv4_attention(e, c.cache, c.table, c.lens_t, z, check=True)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)


def test_page_offsets_beyond_32_bits(ra):
    """Pages that lie more than 2^32 bytes into the cache."""
    page, H, d = 64, 8, 128
    N = (5 << 30) // (page * H * d * 9 // 8)
    cache = ra.Kv4Cache(N, page, H, d)
    rng = np.random.default_rng(77)
    L = 200
    ids = [N - 1, 3, N - 5, N // 2]
    k, v = bf16(rng, L, H, d), bf16(rng, L, H, d)
    t = np.arange(L)
    slots = torch.tensor(np.array(ids)[t // page] * page + t % page).cuda()
    ra.kv4_store(cache, k.cuda(), v.cuda(), slots)
    np.testing.assert_array_equal(f64(ra.kv4_load(cache, slots)[1]), O.rounded(f64(v)))
    c = Case(ra, 77, [0], [1], 16, 8, d, page)
    c.cache, c.lens, c.lens_t = cache, [L], torch.tensor([L], dtype=torch.int32).cuda()
    c.table = torch.tensor([ids], dtype=torch.int32).cuda()
    c.keys, c.values = [O.rounded(f64(k))], [O.rounded(f64(v))]
    c.check(ra, max_q_len=1)


# ------------------------------------------------------------------ use

def test_other_streams_and_two_workspaces(ra):
    a, b = (Case(ra, s, [900, 300], [1, 1], 8, 2, 128, 64) for s in (51, 52))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        outs = []
        for c, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                q = c.q.cuda()
                outs.append(ra.kv4_attention(q, c.cache, c.table, c.lens_t, c.cu_t, o_fp32=True, max_q_len=1))
        torch.cuda.synchronize()
    for c, (o, lse) in zip((a, b), outs):
        want, wl = O.attention(f64(c.q), c.keys, c.values, c.lens, c.cu, True, 1 / math.sqrt(128))
        c.compare(f64(o), f64(lse), want, wl, 1 / math.sqrt(128), True)


def test_sliced_block_table(ra):
    """Rows further apart than they are long; rows without distance are refused."""
    c = Case(ra, 91, [100, 60, 7], [1, 40, 2], 4, 1, 128, 16)
    wide = torch.full((3, c.table.shape[1] + 9), 2 ** 30, dtype=torch.int32).cuda()
    wide[:, 4:4 + c.table.shape[1]] = c.table
    c.table = wide[:, 4:4 + c.table.shape[1]]
    c.check(ra, max_q_len=40)
    c.check(ra, max_q_len=1)
    with pytest.raises(ra.RingAttnError, match="stride"):
        ra.kv4_attention(c.q.cuda(), c.cache, c.table[:1].expand(3, -1), c.lens_t, c.cu_t)
    with pytest.raises(ValueError, match="shape"):
        ra.kv4_attention(c.q.cuda(), c.cache, c.table[:2], c.lens_t, c.cu_t)


def test_captured_prompt_parts_follow_their_lengths(ra):
    """One captured call over other lengths and offsets: what the row-tile kernel and the other one take changes."""
    lens = [300, 500, 40]
    a, b = Case(ra, 92, lens, [100, 1, 30], 4, 2, 128, 16), Case(ra, 93, lens, [3, 120, 8], 4, 2, 128, 16)
    q, table, lens_t, cu = (t.clone() for t in (a.q.cuda(), a.table, a.lens_t, a.cu_t))
    pages = a.cache.pages.clone()
    out = torch.zeros(131, 4, 128).cuda(), torch.zeros(4, 131).cuda()
    ws = ra.kv4_attention_workspace(a.cache, 131, 4, 131)
    call = lambda: ra.kv4_attention(q, a.cache, table, lens_t, cu, o_fp32=True, max_q_len=131, workspace=ws, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in (b, a, b):
        q.copy_(c.q), table.copy_(c.table), lens_t.copy_(c.lens_t), cu.copy_(c.cu_t)
        a.cache.pages.copy_(b.cache.pages if c is b else pages)
        graph.replay()
        ra.kv4_status(ws)
        want, wl = O.attention(f64(c.q), c.keys, c.values, c.lens, c.cu, True, 1 / math.sqrt(128))
        c.compare(f64(out[0]), f64(out[1]), want, wl, 1 / math.sqrt(128), True)


def test_one_workspace_for_calls_of_different_kinds(ra):
    """Its counters are ready for the next call whatever the one before was."""
    ws = ra.kv4_attention_workspace(Case(ra, 1, [5], [1], 8, 1, 128, 16).cache, 200, 8, 200)
    cases = [(Case(ra, 81, [3000, 40], [1, 1], 8, 1, 128, 32), 1), (Case(ra, 82, [900, 500], [100, 2], 8, 1, 128, 32), 100),
             (Case(ra, 83, [2500], [1], 2, 1, 64, 16), 1), (Case(ra, 84, [1800, 90], [3, 1], 8, 1, 128, 64), 3),
             (Case(ra, 85, [4000], [1], 4, 2, 256, 64), 1), (Case(ra, 86, [700], [130], 1, 1, 64, 16), 130)]
    for _ in range(2):
        for c, longest in cases:
            sc = 1 / math.sqrt(c.d)
            o, lse = ra.kv4_attention(c.q.cuda(), c.cache, c.table, c.lens_t, c.cu_t, o_fp32=True, max_q_len=longest,
                                      workspace=ws, check=True)
            want, wl = O.attention(f64(c.q), c.keys, c.values, c.lens, c.cu, True, sc)
            c.compare(f64(o), f64(lse), want, wl, sc, True)


def test_results_repeat(ra):
    c = Case(ra, 61, [3000, 17, 500], [2, 1, 3], 8, 2, 128, 32)
    q = c.q.cuda()
    first = ra.kv4_attention(q, c.cache, c.table, c.lens_t, c.cu_t, o_fp32=True, max_q_len=3)
    for _ in range(4):
        again = ra.kv4_attention(q, c.cache, c.table, c.lens_t, c.cu_t, o_fp32=True, max_q_len=3)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_prompt_then_tokens_in_a_captured_step(ra):
    """Prompts by ring attention, their keys and values into the cache, then decode steps replayed from a CUDA
    graph; a request leaves and another takes its pages."""
    rng = np.random.default_rng(71)
    Hq, Hkv, d, page, R, W = 8, 2, 128, 16, 3, 12
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    N = 20
    cache = ra.Kv4Cache(N, page, Hkv, d)
    table, free, count = torch.full((R, W), -1, dtype=torch.int32).cuda(), torch.arange(N, dtype=torch.int32).cuda(), i32([N])
    lens = i32([0, 0, 0])
    prompt = [37, 1, 64]
    T = sum(prompt)
    q, k, v = bf16(rng, T, Hq, d).cuda(), bf16(rng, T, Hkv, d).cuda(), bf16(rng, T, Hkv, d).cuda()
    out = ra.kv4_tables_out(R, T)._replace(kv_lens=lens, free_count=count)
    step = ra.kv4_tables(lens, i32(prompt), table, page, T, free, count, out=out, check=True)
    cu = step.cu_new.tolist()
    ra.kv4_store(cache, k, v, step.slot_map)
    # the prompt's attention over what the cache holds, by ring attention and by the cache's own
    kr, vr = ra.kv4_load(cache, step.slot_map)
    o_ring, lse_ring = ra.ring_attn_fwd(q, kr, vr, cu, 1, o_fp32=True, check=True)
    o_kv4, lse_kv4 = ra.kv4_attention(q, cache, table, lens, step.cu_new, o_fp32=True, max_q_len=max(prompt), check=True)
    # the ring's P is bf16 (2^-8), the cache's fp16 (2^-11)
    assert (o_ring - o_kv4).abs().max() <= vr.float().abs().max() * (2.0 ** -8 + 2.0 ** -10)
    assert (lse_ring - lse_kv4).abs().max() <= 1e-3

    hist_k = [O.rounded(f64(k[cu[r]:cu[r + 1]])) for r in range(R)]
    hist_v = [O.rounded(f64(v[cu[r]:cu[r + 1]])) for r in range(R)]
    new = i32([1, 1, 1])
    q1, k1, v1 = (torch.zeros(R, h, d, dtype=torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    st = ra.kv4_tables_out(R, R)._replace(kv_lens=lens, free_count=count)
    res = torch.zeros(R, Hq, d).cuda(), torch.zeros(Hq, R).cuda()
    ws = ra.kv4_attention_workspace(cache, R, Hq, 1)

    def one_step():
        ra.kv4_tables(lens, new, table, page, R, free, count, out=st)
        ra.kv4_store(cache, k1, v1, st.slot_map)
        ra.kv4_attention(q1, cache, table, lens, st.cu_new, o_fp32=True, max_q_len=1, workspace=ws, out=res)

    saved = [t.clone() for t in (lens, table, free, count, cache.pages)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one_step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_step()
    for t, s in zip((lens, table, free, count, cache.pages), saved):
        t.copy_(s)
    for i in range(40):
        adds = [1, 1, 1]
        if i == 20:
            adds[2] = -1                                         # the third request leaves ...
        if i == 21:
            adds[2] = 1                                          # ... and its row starts again with one token
        new.copy_(i32(adds))
        n = sum(a > 0 for a in adds)
        qs, ks, vs = bf16(rng, R, Hq, d), bf16(rng, R, Hkv, d), bf16(rng, R, Hkv, d)
        q1.copy_(qs), k1.copy_(ks), v1.copy_(vs)
        graph.replay()
        ra.kv4_status(st.status)
        ra.kv4_status(ws)
        row = 0
        for r, a in enumerate(adds):
            if a < 0:
                hist_k[r], hist_v[r] = hist_k[r][:0], hist_v[r][:0]
            else:
                hist_k[r] = np.concatenate([hist_k[r], O.rounded(f64(ks[row:row + 1]))])
                hist_v[r] = np.concatenate([hist_v[r], O.rounded(f64(vs[row:row + 1]))])
                row += 1
        assert lens.tolist() == [len(x) for x in hist_k]
        if i % 5 == 0 or i in (20, 21, 22):
            cuq = st.cu_new.tolist()
            want, wl = O.attention(f64(qs[:n]), hist_k, hist_v, lens.tolist(), cuq, True, 1 / math.sqrt(d))
            err = np.abs(f64(res[0][:n]) - want).max()
            assert err <= 2.0 ** -10 * max(np.abs(x).max() for x in hist_v if x.size)
            assert np.abs(f64(res[1][:, :n]) - wl).max() <= 1e-4
    used = [p for r in range(R) for p in table[r, :-(-len(hist_k[r]) // page)].tolist()]
    assert sorted(used + free[:int(count)].tolist()) == list(range(N))


# ------------------------------------------------------------------ many units a CTA

def by_heads(c, causal, scale):
    """O.attention's formula, a head's rows at once (many rows)."""
    T = c.cu[-1]
    o, lse = np.zeros((T, c.Hq, c.d)), np.full((c.Hq, T), -np.inf)
    q, G = f64(c.q), c.Hq // c.Hkv
    for r, (L, n) in enumerate(zip(c.lens, c.qlens)):
        if L == 0 or n == 0:
            continue
        b = slice(c.cu[r], c.cu[r + 1])
        see = (L - n + 1 + np.arange(n)).clip(0, L) if causal else np.full(n, L)
        hidden = np.arange(L)[None] >= see[:, None]
        for h in range(c.Hq):
            s = scale * (q[b, h] @ c.keys[r][:, h // G].T)
            s[hidden] = -np.inf
            m = s.max(-1, keepdims=True)
            p = np.exp(s - np.where(np.isneginf(m), 0, m))
            z = p.sum(-1, keepdims=True)
            with np.errstate(divide="ignore"):
                v = c.values[r][:, h // G]
                o[b, h] = (p / np.where(z == 0, 1, z)) @ np.nan_to_num(v)
                o[b, h][(~hidden).astype(np.float64) @ np.isnan(v) > 0] = np.nan   # (a hidden NaN times 0 is none)
                lse[h, b] = (m + np.log(z))[:, 0]
    return o, lse


def test_by_heads_is_the_same_formula(ra):
    c = Case(ra, 5, [30, 0, 5, 64], [7, 2, 9, 64], 4, 2, 64, 16)
    for causal in (True, False):
        for a, b in zip(by_heads(c, causal, 0.2), O.attention(f64(c.q), c.keys, c.values, c.lens, c.cu, causal, 0.2)):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-13)


def run_units(ra, c, longest, causal=True, o_fp32=True):
    """Twice, with one workspace: the formula's values, bit by bit the same."""
    sc = 1 / math.sqrt(c.d)
    want, wl = by_heads(c, causal, sc)
    q = c.q.cuda()
    ws = ra.kv4_attention_workspace(c.cache, c.cu[-1], c.Hq, longest)
    outs = [ra.kv4_attention(q, c.cache, c.table, c.lens_t, c.cu_t, causal=causal, o_fp32=o_fp32, max_q_len=longest,
                             workspace=ws, check=True) for _ in range(2)]
    c.compare(f64(outs[0][0]), f64(outs[0][1]), want, wl, sc, o_fp32)
    assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(*outs))


MIXED = [(40 + 45 * i, 40 + 45 * i if i % 3 == 0 else (1, 7, 130)[i % 3] if i % 2 else 33) for i in range(24)]


@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", [
    (128, 32, 32, [256] * 32, [256] * 32),                       # whole units of 1 and 2 key tiles
    (128, 32, 8, [900] * 16, [280] * 16),                        # the last row tile has 96 rows: an empty second Q tile
    (64, 32, 8, [600] * 64, [90] * 64),
    (128, 32, 8, [a for a, _ in MIXED], [b for _, b in MIXED]),  # prompts, parts of prompts, few rows and single tokens
    (64, 16, 4, [a for a, _ in MIXED], [b for _, b in MIXED]),
    (256, 16, 2, [a for a, _ in MIXED], [b for _, b in MIXED])])
def test_many_prompt_parts(ra, d, Hq, Hkv, lens, qlens):
    """Several units of the row-tile kernel a CTA: phases, notes and tiles carried from one to the next."""
    c = Case(ra, d + len(lens), lens, qlens, Hq, Hkv, d, 32)
    run_units(ra, c, max(qlens))


def test_many_prompt_parts_without_causal_mask(ra):
    c = Case(ra, 95, [a for a, _ in MIXED], [b for _, b in MIXED], 8, 4, 128, 64)
    run_units(ra, c, 1075, causal=False, o_fp32=False)


@pytest.mark.parametrize("d,Hq,Hkv,R,rows", [(64, 2, 1, 700, 50), (128, 8, 8, 300, 1), (64, 4, 1, 1100, 3), (256, 2, 2, 200, 2)])
def test_more_requests_than_threads(ra, d, Hq, Hkv, R, rows):
    rng = random.Random(R)
    lens = [rng.choice([0, 1, 17, 64, rng.randrange(200)]) for _ in range(R)]
    c = Case(ra, R, lens, [rows if i % 5 else 0 for i in range(R)], Hq, Hkv, d, 16)
    run_units(ra, c, rows)


# ------------------------------------------------------------------ rows that are not numbers

def check_broken(ra, c, q, longest, causal=True):
    """Query rows q instead of the case's own, which give the tolerance of the rows that stay numbers."""
    sc = 1 / math.sqrt(c.d)
    good, c.q = c.q, q
    with np.errstate(invalid="ignore"):
        want, wl = O.attention(f64(q), c.keys, c.values, c.lens, c.cu, causal, sc)
    o, lse = ra.kv4_attention(q.cuda(), c.cache, c.table, c.lens_t, c.cu_t, causal=causal, o_fp32=True,
                              max_q_len=longest, check=True)
    c.q = good
    c.compare(f64(o), f64(lse), want, wl, sc, True)
    return want, wl


# few rows and row tiles; whole units, and units split over CTAs (long requests)
ROWS = [(64, 2, 1, [17, 150, 1], [3, 5, 1]), (128, 4, 2, [17, 33, 1000, 0], [1, 2, 5, 3]), (256, 2, 1, [49, 200], [2, 9]),
        (128, 4, 1, [4001], [1]), (256, 4, 1, [2500], [1])]
TILES = [(64, 2, 1, [3001], [70]), (128, 4, 1, [128 * 39 + 1], [30]), (128, 8, 1, [1111, 5], [129, 7]), (256, 4, 1, [2500], [31]),
         (128, 8, 8, [260] * 40, [100] * 40), (256, 8, 2, [130] * 80, [60] * 80)]


@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", ROWS + TILES)
def test_nan_query_rows(ra, d, Hq, Hkv, lens, qlens):
    """A NaN in a query row: NaN in its output and LSE, and in no other row's."""
    c = Case(ra, 101 + d, lens, qlens, Hq, Hkv, d, 16)
    q = c.q.clone()
    rows = list(range(0, c.cu[-1], 3))
    for i in rows:
        q[i, i % Hq, (7 * i) % d] = float("nan")
    want, wl = check_broken(ra, c, q, max(qlens))
    assert np.isnan(want).any() and np.isnan(wl).sum() == sum(not np.isneginf(wl[i % Hq, i]) for i in rows)


@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", [x for x in ROWS + TILES if len(x[3]) < 10])
def test_nan_newest_key(ra, d, Hq, Hkv, lens, qlens):
    """The newest key is NaN: alone in its tile (and part) in some cases, and the last row's score there the only one."""
    rng = np.random.default_rng(3)
    keys = []
    for L in lens:
        k = bf16(rng, L, Hkv, d)
        if L:
            k[L - 1, 0, 5] = float("nan")
        keys.append(k)
    c = Case(ra, 103 + d, lens, qlens, Hq, Hkv, d, 16, keys=keys)
    want, wl = check_broken(ra, c, c.q, max(qlens))
    assert np.isnan(wl).any()
    check_broken(ra, c, c.q, max(qlens), causal=False)


@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", ROWS + TILES)
def test_infinite_queries(ra, d, Hq, Hkv, lens, qlens):
    """An infinity in a query row: every score is infinite or NaN and the softmax has no value, also where all are -inf."""
    rng = np.random.default_rng(4)
    keys = []
    for L in lens:
        k = bf16(rng, L, Hkv, d)
        k[:, :, 3] = 4.0                                         # no code is 0 there
        keys.append(k)
    c = Case(ra, 107 + d, lens, qlens, Hq, Hkv, d, 16, keys=keys)
    q = c.q.clone()
    rows = list(range(0, c.cu[-1], 2))
    for i in rows:
        q[i, i % Hq, 3 if i % 4 else 9] = float("-inf") if i % 3 else float("inf")
    _, wl = check_broken(ra, c, q, max(qlens))
    assert np.isnan(wl).sum() == sum(not np.isneginf(wl[i % Hq, i]) for i in rows)


@pytest.mark.parametrize("n", [3, 70])                           # both kernels
def test_scores_that_vanish(ra, n):
    """A scale times a row's own power of two below the smallest number: equal weights for the keys a row sees."""
    c = Case(ra, 109, [200], [n], 2, 1, 128, 16)
    c.q = (c.q.float() * 2.0 ** -120).to(torch.bfloat16)
    for scale in (1e-30, 1e-8, 1.0):
        c.check(ra, scale=scale, max_q_len=n)


def test_status_words(ra):
    """A wait that was given up has a word above every other one (the largest wins), and names its site."""
    for word, status, text in ((1001, 1, "page"), (1006, 1, "free count"), (2130, 5, "site 130)"), (2150, 5, "site 150)")):
        with pytest.raises(ra.RingAttnError, match=text.replace(")", r"\)")) as e:
            ra.kv4_status(torch.tensor([word, 0], dtype=torch.int32).cuda())
        assert e.value.status == status
    ra.kv4_status(torch.zeros(1, dtype=torch.int32).cuda())


@pytest.mark.parametrize("n", [1, 100])                          # both kernels
def test_the_largest_status_wins(ra, n):
    """Pages outside the cache in every CTA's part, and a request with a length out of range: the status is the length's."""
    cache = ra.Kv4Cache(4, 16, 1, 128)
    L = 600000
    table = torch.full((2, L // 16), -1, dtype=torch.int32).cuda()
    lens = torch.tensor([L, -1], dtype=torch.int32).cuda()
    cu = torch.tensor([0, n, n + 1], dtype=torch.int32).cuda()
    q = torch.ones(n + 1, 1, 128, dtype=torch.bfloat16).cuda()
    ws = ra.kv4_attention_workspace(cache, n + 1, 1, n)
    o, lse = ra.kv4_attention(q, cache, table, lens, cu, max_q_len=n, workspace=ws)
    with pytest.raises(ra.RingAttnError, match="length"):
        ra.kv4_status(ws)
    assert o.eq(0).all() and torch.isneginf(lse).all()


def test_free_count_of_a_step_that_only_maps(ra):
    """Without a free list the count is the caller's, or 0: never what the memory held."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    for count, want in ((None, 0), (i32([5]), 5)):
        out = ra.kv4_tables_out(2, 8)
        for t in out:
            t.fill_(-77)
        step = ra.kv4_tables(i32([3, 0]), i32([1, 4]), i32([[2], [1]]), 16, 8, free_count=count, out=out, check=True)
        assert int(step.free_count) == want
        assert step.slot_map.tolist() == [35, 16, 17, 18, 19, -1, -1, -1]


@pytest.mark.parametrize("big", [0, 20000])                      # one CTA, and many
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_that_are_none_are_reported(ra, big, in_place):
    """A negative page that is given back, taken, or holds a request's last tokens: the step is made, and its status says so."""
    W = big // 16 + 4
    row = lambda *ids: list(ids) + [-9] * (W - len(ids))
    base = dict(lens=[10, 20, 32, 0], new=[1, -1, 2, big], table=[row(0), row(1, 2), row(3, 4), row()],
                free=list(range(10, 10 + W + 2)) + [-5, -5])
    count = W + 2

    def status(want, **change):
        a = {**base, **change}
        slots = sum(max(n, 0) for n in a["new"]) + 3
        got = run_tables(ra, a["lens"], a["new"], a["table"], 16, slots, a["free"], count, in_place)
        assert got == (want,) + O.tables(a["lens"], a["new"], a["table"], 16, slots, a["free"], count)
    status(0)
    status(1001, table=[row(0), row(1, -4), row(3, 4), row()])   # given back
    status(1001, table=[row(-1), row(1, 2), row(3, 4), row()])   # the page of the newest tokens
    status(0, table=[row(0), row(1, 2), row(-1, 4), row()])      # full pages are not looked at
    status(1001, new=[1, 0, 2, big], free=base["free"][:W + 1] + [-1, -5, -5])   # taken


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 8, 8), (128, 8, 8), (128, 8, 2), (256, 8, 4)])
def test_notes_of_many_units(ra, d, Hq, Hkv):
    """NaN values, and pages outside the cache, in some of many units: noted for those alone."""
    rng = np.random.default_rng(d + Hkv)
    lens, qlens = [150 + 13 * (i % 11) for i in range(48)], [100 + i % 3 for i in range(48)]
    values = []
    for i, L in enumerate(lens):
        v = bf16(rng, L, Hkv, d)
        if i % 3 == 1:
            v[L - 1 - 7 * (i % 5), i % Hkv, (5 * i) % d] = float("nan")
        values.append(v)
    c = Case(ra, 111 + d, lens, qlens, Hq, Hkv, d, 16, values=values)
    run_units(ra, c, max(qlens))
    keys = list(c.keys)
    for i in range(0, 48, 4):                                    # keys 16 to 31 of every fourth request are left out
        c.table[i, 1] = -1
        keys[i], c.values[i] = (np.delete(x, np.s_[16:32], axis=0) for x in (c.keys[i], c.values[i]))
    ws = ra.kv4_attention_workspace(c.cache, c.cu[-1], Hq, max(qlens))
    o, lse = ra.kv4_attention(c.q.cuda(), c.cache, c.table, c.lens_t, c.cu_t, o_fp32=True, max_q_len=max(qlens), workspace=ws)
    with pytest.raises(ra.RingAttnError, match="page"):
        ra.kv4_status(ws)
    c.keys, c.lens = keys, [len(k) for k in keys]
    want, wl = by_heads(c, True, 1 / math.sqrt(d))
    c.compare(f64(o), f64(lse), want, wl, 1 / math.sqrt(d), True)


def test_streams_and_graphs_over_many_units(ra):
    """Two calls at once, each with its own workspace: eager on two streams, and two captured graphs replayed together."""
    cs = [Case(ra, s, [a for a, _ in MIXED], [b for _, b in MIXED], 8, 4, 128, 32) for s in (121, 122)]
    T = cs[0].cu[-1]
    qs, wss = [c.q.cuda() for c in cs], [ra.kv4_attention_workspace(c.cache, T, 8, 1075) for c in cs]
    outs = [(torch.zeros(T, 8, 128).cuda(), torch.zeros(8, T).cuda()) for _ in cs]
    wants = [by_heads(c, True, 1 / math.sqrt(128)) for c in cs]
    call = lambda i: ra.kv4_attention(qs[i], cs[i].cache, cs[i].table, cs[i].lens_t, cs[i].cu_t, o_fp32=True,
                                      max_q_len=1075, workspace=wss[i], out=outs[i])
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    graphs = []
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            for _ in range(4):
                call(i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)

    def check():
        torch.cuda.synchronize()
        for c, w, (o, lse), (want, wl) in zip(cs, wss, outs, wants):
            ra.kv4_status(w)
            c.compare(f64(o), f64(lse), want, wl, 1 / math.sqrt(128), True)
            o.zero_(), lse.zero_()
        torch.cuda.synchronize()
    check()
    for run in (call, lambda i: graphs[i].replay()):
        for _ in range(5):
            for i, st in enumerate(streams):
                with torch.cuda.stream(st):
                    run(i)
        check()


@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", [
    (64, 600, 300, [100, 33], [2, 1]), (128, 4096, 1, [70, 40], [3, 1]), (128, 300, 300, [200, 100], [110, 1]),
    (64, 2, 1, [60 + i % 50 for i in range(5000)], [50 if i % 7 == 0 else 1 for i in range(5000)])])
def test_many_heads_and_requests(ra, d, Hq, Hkv, lens, qlens):
    run_units(ra, Case(ra, Hq, lens, qlens, Hq, Hkv, d, 16), max(qlens))


@pytest.mark.parametrize("d,n,log", [(64, 1, 27), (128, 1, 28), (64, 100, 26)])
def test_very_long_request(ra, d, n, log):
    """2^26 to 2^28 cached tokens (a table that repeats seven pages).  An accumulator takes the L / (16 x 152) tiles of 16
    keys of its part at most, each addition off by at most 2^-23 of the sum, in o and in l."""
    rng = np.random.default_rng(log)
    page, P, L = 256, 7, 1 << log
    cache = ra.Kv4Cache(P, page, 1, d)
    k, v = bf16(rng, P * page, 1, d), bf16(rng, P * page, 1, d)
    ra.kv4_store(cache, k.cuda(), v.cuda(), torch.arange(P * page).cuda())
    k, v = O.rounded(f64(k))[:, 0], O.rounded(f64(v))[:, 0]
    table = (torch.arange(L // page, device="cuda") % P).int()[None]
    q = bf16(rng, n, 1, d)
    o, lse = ra.kv4_attention(q.cuda(), cache, table, torch.tensor([L], dtype=torch.int32).cuda(),
                              torch.tensor([0, n], dtype=torch.int32).cuda(), causal=False, o_fp32=True, max_q_len=n, check=True)
    times = np.array([(L // page - p + P - 1) // P for p in range(P)]).repeat(page)
    s = f64(q)[:, 0] @ k.T / math.sqrt(d)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m) * times
    z = w.sum(1, keepdims=True)
    e_s = math.sqrt(d) * 2.0 ** -23 * np.abs(f64(q)).max() * np.abs(k).sum(-1).max()
    e = L / (16 * 152) * 2.0 ** -23 + 2.0 ** -11 + 2.0 ** -20 + 2 * e_s
    assert np.abs(f64(o)[:, 0] - (w / z) @ v).max() <= 2 * e * np.abs(v).max()
    assert np.abs(f64(lse)[0] - (m + np.log(z))[:, 0]).max() <= e
