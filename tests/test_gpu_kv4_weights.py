"""Attention weights of cached tokens on the GPU against the fp64 oracle.

Tolerance of a sum, relative to it: the exponent's error (S in fp32 from exact
products, as for cache attention: D terms, each off by at most one unit in the
last place, 2^-23, of the sum of magnitudes; its scaling and the log-sum-exp's, 2^-22
of their sizes), 2^x (2^-20), and the additions (at most N terms: N 2^-23); beside it
2^-126 for each term that underflows.
"""

import math

import numpy as np
import pytest
import torch

from oracle import kv4 as O
from oracle import kv4_evict as E

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


class Case:
    """A cache with random pages, the keys of several requests in it, query rows and sums that hold something."""

    def __init__(self, ra, seed, lens, qlens, Hq, Hkv, d, page, kscale=1.0, garbage=True, keys=None, spare=2):
        rng = np.random.default_rng(seed)
        self.lens, self.qlens, self.Hq, self.Hkv, self.d, self.page = lens, qlens, Hq, Hkv, d, page
        held = [-(-n // page) for n in lens]
        self.N = N = sum(held) + spare
        ids = rng.permutation(N)
        table = np.full((len(lens), max(held + [0]) + 2), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(held):
            table[r, :n] = ids[at:at + n]
            at += n
        self.cache = ra.Kv4Cache(N, page, Hkv, d)
        if garbage:   # what unused places hold must not matter: all bytes, NaN scales among them
            self.cache.pages.random_(0, 256, generator=torch.Generator("cuda").manual_seed(seed))
        self.keys, self.slots = [], []
        for r, n in enumerate(lens):
            k = torch.tensor(rng.standard_normal((n, Hkv, d)) * kscale, dtype=torch.float32).to(torch.bfloat16)
            k = k if keys is None else keys[r]
            t = np.arange(n)
            slots = table[r, t // page].astype(np.int64) * page + t % page
            ra.kv4_store(self.cache, k.cuda(), torch.zeros_like(k).cuda(), torch.tensor(slots).cuda())
            self.keys.append(O.rounded(f64(k)))
            self.slots.append(slots)
        self.cu = np.concatenate([[0], np.cumsum(qlens)]).astype(int).tolist()
        self.q = torch.tensor(rng.standard_normal((self.cu[-1], Hq, d)), dtype=torch.float32).to(torch.bfloat16)
        self.table, self.lens_t, self.cu_t = torch.tensor(table).cuda(), i32(lens), i32(self.cu)
        self.before = torch.tensor(rng.exponential(size=N * page), dtype=torch.float32)
        self.new = [int(rng.integers(-1, n + 3)) for n in lens]

    def lse(self, ra, causal=True, scale=None):
        return ra.kv4_attention(self.q.cuda(), self.cache, self.table, self.lens_t, self.cu_t, causal=causal,
                                scale=scale)[1]

    def run(self, ra, lse, causal=True, scale=None, new=True, q=None, **kw):
        w = self.before.cuda()
        got = ra.kv4_weights(self.q.cuda() if q is None else q, self.cache, self.table, self.lens_t, self.cu_t, lse, w,
                             new_lens=i32(self.new) if new else None, causal=causal, scale=scale, **kw)
        assert got is w
        return w

    def check(self, ra, causal=True, scale=None, lse=None, **kw):
        lse = self.lse(ra, causal, scale) if lse is None else lse
        for new in (True, False):
            w = self.run(ra, lse, causal, scale, new, check=True, **kw)
            self.compare(w, lse, causal, scale, new)
        return w

    def compare(self, w, lse, causal=True, scale=None, new=True):
        sc = scale or 1 / math.sqrt(self.d)
        q, z, got, want = f64(self.q), f64(lse), f64(w), f64(self.before)
        sums = E.weights(q, self.keys, self.lens, self.cu, z, causal, sc)
        tol = np.zeros(len(want))
        finite = z[np.isfinite(z)]
        zmax = np.abs(finite).max() if finite.size else 0.0
        fq = np.where(np.isfinite(q), q, 0.0)
        for r, L in enumerate(self.lens):
            if L == 0:
                continue
            fresh = L - min(max(self.new[r], 0), L) if new else L
            begin = want[self.slots[r]]
            begin[fresh:] = 0.0
            rows = fq[self.cu[r]:self.cu[r + 1]]
            k = np.nan_to_num(np.abs(self.keys[r]))
            ks, qm = k.sum(-1).max(), (np.abs(rows).max() if rows.size else 0.0)
            n = rows.shape[0] * self.Hq
            xmax = sc * qm * ks
            rel = sc * self.d * 2.0 ** -23 * qm * ks + (min(xmax, 200) + zmax) * 2.0 ** -22 + 2.0 ** -20 + (n + 2) * 2.0 ** -23
            want[self.slots[r]] = begin + sums[r]
            tol[self.slots[r]] = rel * np.nan_to_num(begin + sums[r]) + n * 2.0 ** -126
        assert np.array_equal(np.isnan(got), np.isnan(want))
        f = ~np.isnan(want)
        assert np.all(np.abs(got[f] - want[f]) <= tol[f]), np.abs(got[f] - want[f]).max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 5, 8, 16])
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(ra, d, G, page):
    lens = [1, 2, 15, 16, 17, 31, 63, 64, 65, 0, 130, 1000]
    Case(ra, 7 * d + G, lens, [1] * len(lens), 2 * G, 2, d, page).check(ra, max_q_len=1)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,Hq,Hkv,qlens", [(64, 4, 2, [3, 0, 7, 1, 5]), (128, 8, 8, [9, 1, 0, 2, 33]), (256, 7, 1, [2, 3, 4, 0, 1]),
                                            (128, 12, 4, [8, 20, 1, 4, 3])])
def test_several_tokens(ra, d, Hq, Hkv, qlens, causal):
    c = Case(ra, d + Hq, [40, 129, 700, 1, 64], qlens, Hq, Hkv, d, 32)
    c.check(ra, causal, max_q_len=max(qlens))
    c.check(ra, causal, scale=0.37, max_q_len=max(qlens))


@pytest.mark.parametrize("d,Hq,Hkv,L", [(64, 2, 2, 40000), (128, 32, 8, 20011), (256, 16, 2, 9001)])
def test_one_long_request(ra, d, Hq, Hkv, L):
    Case(ra, L, [L], [1], Hq, Hkv, d, 64).check(ra)


def test_more_rows_than_keys(ra):
    """The first query tokens of such a request see no key; their log-sum-exp is -inf."""
    c = Case(ra, 3, [5, 1], [9, 4], 4, 2, 128, 16)
    lse = c.lse(ra)
    assert torch.isneginf(lse[:, :4]).all()
    c.check(ra, lse=lse)


@pytest.mark.parametrize("d,Hq,Hkv,n", [(128, 40, 40, 1), (64, 96, 96, 2), (256, 28, 14, 5), (128, 64, 1, 3), (128, 24, 2, 7)])
def test_more_rows_than_shared_memory_holds(ra, d, Hq, Hkv, n):
    """Heads, or row tiles of one head, by turns."""
    Case(ra, Hq + n, [300, 77, 1000], [n, 1, n], Hq, Hkv, d, 32).check(ra, max_q_len=n)


def test_many_requests(ra):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    qlens = [int(min(n, x)) for n, x in zip(lens, rng.integers(0, 3, 700))]
    Case(ra, 17, lens, qlens, 4, 2, 64, 16).check(ra, max_q_len=2)


def test_sums_of_a_step_without_rows(ra):
    """Only the new tokens' sums change, to zero; with no request, or no rows at all, too."""
    c = Case(ra, 8, [100, 33, 0, 64], [0, 0, 0, 0], 4, 2, 64, 16)
    lse = torch.empty(4, 0).cuda()
    c.new = [40, -1, 0, 64]
    c.check(ra, lse=lse)
    w = c.before.cuda()
    ra.kv4_weights(c.q.cuda(), c.cache, c.table[:0], c.lens_t[:0], c.cu_t[:1], lse, w, check=True)
    assert torch.equal(w.cpu(), c.before)


def test_layers_share_sums(ra):
    """Two layers in turn: the second one adds."""
    a = Case(ra, 11, [70, 200], [1, 2], 8, 2, 64, 16)
    lse = a.lse(ra)
    once = a.run(ra, lse)
    a.before = once.cpu()
    a.compare(a.run(ra, lse, new=False), lse, new=False)


def test_masked_rows_and_keys_that_are_no_numbers(ra):
    """A NaN row makes the sums NaN of the keys it sees and of no others; a NaN key its own."""
    lens, qlens = [100, 50, 64], [3, 2, 4]
    rng = np.random.default_rng(2)
    keys = [torch.tensor(rng.standard_normal((n, 2, 64)), dtype=torch.float32).to(torch.bfloat16) for n in lens]
    keys[1][49, 1, 3] = float("nan")                             # the newest token: seen by the last row alone
    keys[1][7, 0, 50] = float("inf")
    c = Case(ra, 2, lens, qlens, 4, 2, 64, 16, keys=keys)
    z = torch.full((4, 9), 3.0).cuda()
    z[2, 0] = float("-inf")                                      # a row without a softmax: adds nothing
    c.q[1, 0, 5] = float("inf")                                  # request 0, row 1: sees 99 keys of 100
    c.q[5, 3, 9] = float("nan")                                  # request 2, row 0: sees 61 of 64
    z[1, 8] = float("nan")                                       # request 2, the last row
    z[0, 4] = float("inf")
    q = f64(c.q)
    want = E.weights(np.where(np.isfinite(q), q, np.nan), c.keys, c.lens, c.cu, f64(z), True, 0.125)
    w = c.run(ra, z, new=False, check=True)
    got = f64(w)
    for r in range(3):
        assert np.array_equal(np.isnan(got[c.slots[r]]), np.isnan(want[r]))
    assert not np.isnan(got[c.slots[0][99]]) and np.isnan(got[c.slots[0][98]])
    assert np.isnan(got[c.slots[1]]).nonzero()[0].tolist() == [7, 49]
    c.q = torch.tensor(np.where(np.isfinite(q), q, np.nan))
    c.compare(w, z, new=False)


def test_large_scores(ra):
    """Uneven and large scores: the weights are those of a softmax still."""
    c = Case(ra, 21, [500, 33], [2, 5], 4, 2, 128, 16, kscale=30.0)
    w = c.check(ra)
    sums = f64(w)[c.slots[0]] - f64(c.before)[c.slots[0]]
    assert abs(sums.sum() - 8) < 1e-2                            # 2 rows x 4 heads: each row's weights add up to one


def test_strided_queries_and_other_slots(ra):
    c = Case(ra, 31, [90, 17], [3, 1], 6, 3, 128, 16, spare=9)
    lse = c.lse(ra)
    wide = torch.randn(4, 14, 128).to(torch.bfloat16).cuda()
    wide[:, 4:10] = c.q.cuda()
    c.check(ra, lse=lse, q=wide[:, 4:10])
    # rows outside [cu[0], cu[R]) belong to no request
    more = torch.cat([c.q.cuda(), torch.full((3, 6, 128), float("nan"), dtype=torch.bfloat16).cuda()])
    z = torch.cat([lse, torch.full((6, 3), float("nan")).cuda()], 1)
    w = c.before.cuda()
    ra.kv4_weights(more, c.cache, c.table, c.lens_t, c.cu_t, z, w, check=True)
    c.compare(w, lse, new=False)


def test_refused_contents_are_reported_and_stay_in_bounds(ra):
    def fresh():
        return Case(ra, 41, [200, 100, 300, 64], [2, 1, 2, 1], 4, 2, 64, 16, spare=3)

    lse = fresh().lse(ra)
    for what, code in (("page", 1), ("far page", 1), ("length", 1), ("long", 1), ("offset", 1), ("end", 1)):
        c = fresh()
        c.new = [0, 0, 0, 0]
        if what == "page":
            c.table[2, 3] = -5
        elif what == "far page":
            c.table[2, 3] = c.N
        elif what == "length":
            c.lens_t[1] = -3
        elif what == "long":
            c.lens_t[1] = (1 << 30) + 5
        elif what == "offset":
            c.cu_t[2] = 1
        else:
            c.cu_t[4] = 7
        guard = torch.full((c.N * c.page + 2048,), 7.5, device="cuda")
        w = guard[1024:1024 + c.N * c.page]
        w.copy_(c.before)
        ws = ra.kv4_attention_workspace(c.cache, 6, 4)
        ra.kv4_weights(c.q.cuda(), c.cache, c.table, c.lens_t, c.cu_t, lse, w, workspace=ws)
        with pytest.raises(ra.RingAttnError) as e:
            ra.kv4_status(ws)
        assert e.value.status == code
        assert torch.all(guard[:1024] == 7.5) and torch.all(guard[-1024:] == 7.5)
        got, ref = f64(w), f64(fresh().run(ra, lse, new=False))
        if "page" in what:                                       # the other 284 tokens' sums are not affected
            skip = c.slots[2][48:64]
            assert np.array_equal(got[skip], f64(c.before)[skip])
            got[skip] = ref[skip]
            assert np.array_equal(got, ref)
        elif what in ("length", "long"):
            assert np.array_equal(got[c.slots[1]], f64(c.before)[c.slots[1]])
            assert np.array_equal(got[c.slots[0]], ref[c.slots[0]]) and np.array_equal(got[c.slots[2]], ref[c.slots[2]])
        else:
            assert np.array_equal(got[c.slots[0]], ref[c.slots[0]])
        ra.kv4_weights(c.q.cuda(), fresh().cache, fresh().table, fresh().lens_t, fresh().cu_t, lse, w, workspace=ws)
        ra.kv4_status(ws)                                        # the next call's status is its own


def test_offsets_beyond_32_bits(ra):
    """A request on the last pages of a cache of more than 2^32 bytes."""
    page, d = 256, 64
    N = (1 << 32) // (256 // 16 * 18 * d) + 900
    cache = ra.Kv4Cache(N, page, 1, d)
    L = 700
    k = torch.randn(L, 1, d).to(torch.bfloat16).cuda()
    table = i32([[N - 1, N - 3, N - 2]])
    t = torch.arange(L).cuda()
    slots = table[0][t // page].long() * page + t % page
    ra.kv4_store(cache, k, k, slots)
    q = torch.randn(2, 2, d).to(torch.bfloat16).cuda()
    lens, cu = i32([L]), i32([0, 2])
    _, lse = ra.kv4_attention(q, cache, table, lens, cu, check=True)
    w = torch.zeros(N * page, device="cuda")
    ra.kv4_weights(q, cache, table, lens, cu, lse, w, check=True)
    assert abs(float(w.double().sum()) - 4) < 1e-4 and int((w != 0).sum()) == L
    want = E.weights(f64(q), [O.rounded(f64(k))], [L], [0, 2], f64(lse), True, 0.125)[0]
    assert np.abs(f64(w[slots]) - want).max() < 1e-6


def test_results_repeat_on_streams_and_in_graphs(ra):
    c = Case(ra, 51, [3000, 77, 900, 16], [1, 2, 1, 1], 16, 4, 128, 32)
    lse, q, new = c.lse(ra), c.q.cuda(), i32(c.new)
    want = c.run(ra, lse, max_q_len=2)
    torch.cuda.synchronize()
    runs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            w = c.before.cuda()
            ra.kv4_weights(q, c.cache, c.table, c.lens_t, c.cu_t, lse, w, new_lens=new, max_q_len=2)
            runs.append(w)
    torch.cuda.synchronize()
    assert all(torch.equal(w, want) for w in runs)
    w, ws, lens = c.before.cuda(), ra.kv4_attention_workspace(c.cache, 5, 16, 2), c.lens_t.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.kv4_weights(q, c.cache, c.table, lens, c.cu_t, lse, w, new_lens=new, max_q_len=2, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want)
    w.copy_(c.before)
    lens[0] = 1234                                               # lengths are read by the kernel
    graph.replay()
    short = c.before.cuda()
    ra.kv4_weights(q, c.cache, c.table, lens, c.cu_t, lse, short, new_lens=new, max_q_len=2)
    torch.cuda.synchronize()
    assert torch.equal(w, short) and not torch.equal(w, want)
    ra.kv4_status(ws)


def test_refusals(ra):
    c = Case(ra, 61, [64, 30], [1, 1], 4, 2, 64, 16)
    lse, q, w = c.lse(ra), c.q.cuda(), c.before.cuda()
    ok = dict(q=q, cache=c.cache, block_table=c.table, kv_lens=c.lens_t, cu_q=c.cu_t, lse=lse, weights=w)
    for kw, word in ((dict(q=q.float()), "dtype"), (dict(q=q[0]), "shape"), (dict(lse=lse.t().contiguous()), "lse"),
                     (dict(lse=lse.double()), "lse"), (dict(weights=w[:-1]), "weights"), (dict(weights=w.cpu()), "weights"),
                     (dict(new_lens=c.lens_t[:1]), "new_lens"), (dict(cu_q=c.cu_t[:2]), "cu_q"),
                     (dict(q=q.float().requires_grad_()), "no gradient")):
        with pytest.raises(ValueError, match=word):
            ra.kv4_weights(**dict(ok, **kw))
    with pytest.raises(ra.RingAttnError, match="lie over"):
        ra.kv4_weights(**dict(ok, weights=c.cache.pages.view(-1).view(torch.float32)[:w.numel()]))
    with pytest.raises(ra.RingAttnError, match="workspace"):
        ra.kv4_weights(**dict(ok, workspace=torch.zeros(128, dtype=torch.uint8, device="cuda")))
    with pytest.raises(ra.RingAttnError, match="multiple"):
        ra.kv4_weights(**dict(ok, q=torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda"), lse=lse[:3].contiguous()))


# ------------------------------------------------------------------ many rows: the tile kernel

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", [
    (128, 8, 2, [300], [40]), (64, 2, 2, [1000], [130]), (256, 4, 2, [700], [50]),
    (128, 15, 3, [257, 900], [33, 100]), (64, 7, 1, [2000, 129, 128], [64, 20, 128]),
    (256, 28, 4, [513, 90], [31, 90]), (128, 32, 8, [5000], [64])])
def test_prompt_parts(ra, d, Hq, Hkv, lens, qlens, causal):
    Case(ra, d + Hq, lens, qlens, Hq, Hkv, d, 32).check(ra, causal, max_q_len=max(qlens))


@pytest.mark.parametrize("d,Hq,Hkv,n", [(128, 160, 1, 3), (256, 130, 2, 2), (64, 129, 1, 1), (256, 65, 1, 4), (128, 127, 1, 5)])
def test_large_groups(ra, d, Hq, Hkv, n):
    """Query tiles that hold a part of one token's heads, or one token and little else."""
    Case(ra, Hq, [400, 90], [n, n], Hq, Hkv, d, 16).check(ra, max_q_len=n)


@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", [(128, 80, 40, [200], [40]), (64, 64, 64, [256, 17], [70, 64]),
                                                 (256, 24, 24, [130], [128]), (128, 16, 16, [1500, 3], [100, 2])])
def test_blocks_of_many_ctas(ra, d, Hq, Hkv, lens, qlens):
    """Few blocks of keys with many heads: their sums come from several CTAs."""
    Case(ra, Hq + d, lens, qlens, Hq, Hkv, d, 64).check(ra, max_q_len=max(qlens))


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 8, 2), (128, 32, 8), (256, 16, 8)])
def test_prompt_parts_among_single_tokens(ra, d, Hq, Hkv):
    lens = [700, 1, 300, 64, 2000, 0, 90, 512]
    qlens = [1, 1, 200, 5, 16, 0, 0, 333]
    c = Case(ra, 9 + d, lens, qlens, Hq, Hkv, d, 64)
    c.check(ra, max_q_len=333)
    c.check(ra, False, max_q_len=333)


def test_many_requests_of_many_rows(ra):
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(1, 700, 300)]
    qlens = [int(min(n, x)) for n, x in zip(lens, rng.integers(0, 120, 300))]
    Case(ra, 27, lens, qlens, 4, 2, 64, 16).check(ra, max_q_len=120)


def test_one_request_without_rows(ra):
    """A call that names a long request and brings none: only the new tokens' sums change."""
    c = Case(ra, 8, [1000], [0], 4, 2, 128, 16)
    c.new = [600]
    w = c.before.cuda()
    z, q = torch.zeros(4, 80).cuda(), torch.zeros(80, 4, 128, dtype=torch.bfloat16).cuda()
    ra.kv4_weights(q, c.cache, c.table, c.lens_t, c.cu_t, z, w, new_lens=i32(c.new), check=True)
    want = c.before.clone()
    want[torch.tensor(c.slots[0][400:])] = 0
    assert torch.equal(w.cpu(), want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_and_keys_that_are_no_numbers_in_tiles(ra, d):
    lens, qlens = [600, 300], [90, 70]
    rng = np.random.default_rng(d)
    keys = [torch.tensor(rng.standard_normal((n, 2, d)), dtype=torch.float32).to(torch.bfloat16) for n in lens]
    keys[0][599, 1, 3] = float("nan")                            # the newest token: seen by the last row alone
    keys[0][17, 0, 50] = float("inf")
    keys[1][299, 0, 0] = float("nan")
    c = Case(ra, 2, lens, qlens, 4, 2, d, 16, keys=keys)
    z = torch.full((4, 160), 3.0).cuda()
    z[2, 0] = z[1, 89] = float("-inf")
    z[3, 159] = float("-inf")                                    # the only rows that see request 1's newest key: those of head 0 to 2
    z[0, 30] = float("nan")                                      # request 0, row 30: sees 541 keys
    c.q[95, 1, 7] = float("nan")                                 # request 1, row 5: sees 236
    q = f64(c.q)
    want = E.weights(q, c.keys, c.lens, c.cu, f64(z), True, 1 / math.sqrt(d))
    w = c.run(ra, z, new=False, check=True)
    for r in range(2):
        assert np.array_equal(np.isnan(f64(w)[c.slots[r]]), np.isnan(want[r]))
    assert np.isnan(want[0]).nonzero()[0].tolist() == list(range(541)) + [599]
    assert np.isnan(want[1]).nonzero()[0].tolist() == list(range(236)) + [299]
    c.compare(w, z, new=False)
    # a request whose rows have no softmax at all adds nothing, whatever its keys are
    z[:, 90:] = float("-inf")
    w = c.run(ra, z, new=False, check=True)
    assert np.array_equal(f64(w)[c.slots[1]], f64(c.before)[c.slots[1]])


def test_bad_pages_lengths_and_offsets_in_tiles(ra):
    def fresh():
        return Case(ra, 43, [800, 100, 900], [70, 1, 80], 4, 2, 64, 16, spare=3)

    lse = fresh().lse(ra)
    ref = f64(fresh().run(ra, lse, new=False, max_q_len=80))
    for what in ("page", "far page", "length", "offset"):
        c = fresh()
        if what == "page":
            c.table[2, 30] = -1
        elif what == "far page":
            c.table[2, 30] = 1 << 30
        elif what == "length":
            c.lens_t[2] = 1 << 20
        else:
            c.cu_t[3] = 200
        w, ws = c.before.cuda(), ra.kv4_attention_workspace(c.cache, 151, 4, 80)
        ra.kv4_weights(c.q.cuda(), c.cache, c.table, c.lens_t, c.cu_t, lse, w, max_q_len=80, workspace=ws)
        with pytest.raises(ra.RingAttnError) as e:
            ra.kv4_status(ws)
        assert e.value.status == 1
        got, want = f64(w), ref.copy()
        if "page" in what:
            want[c.slots[2][480:496]] = f64(c.before)[c.slots[2][480:496]]
        else:
            want[c.slots[2]] = f64(c.before)[c.slots[2]]
        assert np.array_equal(got, want)
        ra.kv4_weights(c.q.cuda(), fresh().cache, fresh().table, fresh().lens_t, fresh().cu_t, lse, w, max_q_len=80, workspace=ws)
        ra.kv4_status(ws)


def test_strided_queries_and_graphs_in_tiles(ra):
    c = Case(ra, 33, [900, 333], [64, 40], 8, 2, 128, 32)
    lse = c.lse(ra)
    wide = torch.randn(104, 12, 128).to(torch.bfloat16).cuda()
    wide[:, 2:10] = c.q.cuda()
    want = c.check(ra, lse=lse, q=wide[:, 2:10], max_q_len=64)
    want = c.run(ra, lse, max_q_len=64)
    q, new, lens, cu = c.q.cuda(), i32(c.new), c.lens_t.clone(), c.cu_t.clone()
    w, ws = c.before.cuda(), ra.kv4_attention_workspace(c.cache, 104, 8, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.kv4_weights(q, c.cache, c.table, lens, cu, lse, w, new_lens=new, max_q_len=64, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want)
    for n0, n1, L in ((1, 3, 500), (0, 0, 0), (30, 40, 901)):    # rows and lengths change between replays
        cu.copy_(i32([0, n0, n0 + n1]))
        lens[0] = L
        w.copy_(c.before)
        graph.replay()
        alone = c.before.cuda()
        ra.kv4_weights(q, c.cache, c.table, lens, cu, lse, alone, new_lens=new, max_q_len=64)
        torch.cuda.synchronize()
        assert torch.equal(w, alone)
        ra.kv4_status(ws)


def test_both_kernels_agree(ra):
    """The same rows by either kernel (max_q_len selects): fp32 sums in another order."""
    c = Case(ra, 71, [3000, 40], [70, 40], 8, 2, 128, 64)
    lse = c.lse(ra)
    a, b = c.run(ra, lse, max_q_len=70), c.run(ra, lse, max_q_len=1)
    c.compare(a, lse)
    c.compare(b, lse)
    assert torch.allclose(a, b, rtol=2e-5, atol=1e-7)


@pytest.mark.parametrize("d,Hq,Hkv,lens,qlens", [
    (64, 2, 2, [40000], [1]), (128, 32, 8, [20011, 300], [1, 2]), (128, 24, 2, [6000, 900], [7, 7]), (256, 16, 2, [9001], [2]),
    (64, 4, 2, [9000, 800, 1], [130, 1, 1]), (128, 8, 2, [9000], [70]), (128, 7, 1, [3000, 700], [40, 50]),
    (256, 4, 1, [5000, 70], [40, 40])])
def test_what_is_added_to_old_sums(ra, d, Hq, Hkv, lens, qlens):
    """A step adds its weights, once, to slots that may hold far more than it adds.

    The tolerance above belongs to the added sums alone; what a slot held is only added to:
    half a step (2^-24) of the result for each of at most Hkv (rows / 64 + 1) + 1 additions."""
    c = Case(ra, 13 * d + lens[0], lens, qlens, Hq, Hkv, d, 64)
    c.new = [0] * len(lens)
    lse = c.lse(ra)
    z, q, before = f64(lse), f64(c.q), f64(c.before)
    sums = E.weights(q, c.keys, c.lens, c.cu, z, True, 1 / math.sqrt(d))
    got = f64(c.run(ra, lse, max_q_len=max(qlens), check=True))
    for r, n in enumerate(qlens):
        rows = n * Hq
        x = np.abs(q[c.cu[r]:c.cu[r + 1]]).max() * np.abs(c.keys[r]).sum(-1).max() / math.sqrt(d)
        rel = d * 2.0 ** -23 * x + (min(x, 200) + np.abs(z[np.isfinite(z)]).max()) * 2.0 ** -22 + 2.0 ** -20 + (rows + 2) * 2.0 ** -23
        old = before[c.slots[r]]
        adds = Hkv * (rows // Hkv // 64 + 1) + 1
        tol = rel * sums[r] + adds * 2.0 ** -24 * (old + sums[r]) + rows * 2.0 ** -126
        assert np.all(np.abs(got[c.slots[r]] - (old + sums[r])) <= tol)
        assert np.median(tol) < np.median(sums[r]) / 4           # (one that is left out, or added twice, shows)
    rest = np.setdiff1d(np.arange(len(before)), np.concatenate([np.array(s) for s in c.slots]))
    assert np.array_equal(got[rest], before[rest])
