"""Attention weights of cached tokens and eviction without a GPU: the oracle's own pins, and what the calls refuse
before any device work."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4_evict as E


# ------------------------------------------------------------------ the oracle's own pins

@pytest.mark.parametrize("causal", [True, False])
def test_weights_add_up_to_the_rows(causal):
    """With the rows' own log-sum-exps a request's weights add up to its rows (that see a key)."""
    rng = np.random.default_rng(5)
    lens, cu, Hq, Hkv, d, scale = [7, 3, 5, 0], [0, 2, 5, 5, 6], 4, 2, 8, 0.3
    q = rng.standard_normal((6, Hq, d))
    keys = [rng.standard_normal((n, Hkv, d)) for n in lens]
    lse = np.full((Hq, 6), -np.inf)
    for r, n in enumerate(lens):
        for i in range(cu[r], cu[r + 1]):
            last = n - (cu[r + 1] - i) if causal else n - 1
            for h in range(Hq):
                x = scale * keys[r][:last + 1, h // 2] @ q[i, h]
                if len(x):
                    lse[h, i] = math.log(np.exp(x).sum())
    got = E.weights(q, keys, lens, cu, lse, causal, scale)
    assert [len(w) for w in got] == lens
    for w, rows in zip(got, (2, 3, 0, 0)):
        assert abs(w.sum() - Hq * rows) < 1e-12
    assert np.all(got[2] == 0)


def test_rows_without_a_softmax_see_no_key():
    q, keys = np.full((1, 1, 2), np.nan), [np.ones((2, 1, 2))]
    assert np.all(E.weights(q, keys, [2], [0, 1], np.full((1, 1), -np.inf), True, 1.0)[0] == 0)
    assert np.all(np.isnan(E.weights(q, keys, [2], [0, 1], np.zeros((1, 1)), True, 1.0)[0]))


def test_eviction_by_hand():
    # pages of 4: tokens 0..9 in slots 8..11, 0..3, 12, 13; the first and the last two stay
    table, w = [[2, 0, 3]], [5, 1, 9, 9, 0, 0, 0, 0, 0, 2, 3, 3, 0, 0, 0, 0]
    out = E.evict(w, table, [10], [6], 4, 4, 1, 2, 1, free=[7, -1, -1], count=1)
    # token      0  1  2  3  4  5  6  7  8  9
    # sum        0  2  3  3  5  1  9  9  0  0: 6, 7 and 4 stay; 6..9 move into places 1, 2, 3 and 5
    assert out[0] == [6] and out[1] == [4]
    assert out[2] == [[2, 3, 12, 13]] and out[3] == [[9, 10, 11, 1]]
    assert out[4] == 2 and out[5] == [7, 3, -1] and out[6] == []
    # of equal sums the lower index stays
    out = E.evict([1.0] * 16, table, [10], [6], 4, 4, 1, 2, 1)
    assert out[2] == [[12, 13, -1, -1]] and out[3] == [[0, 1, -1, -1]]
    # within budget and slack, or without a budget: nothing
    for L, B, slack in ((7, 6, 1), (10, -1, 0), (0, 0, 0)):
        out = E.evict(w, table, [L], [B], 4, 4, slack, 1, 1)
        assert out[0] == [L] and out[1] == [0] and out[2] == [[-1] * 4] and out[6] == []
    # cannot be cut: too long for the table, a budget below what is protected, a page that is none, too many moves
    for L, B, tab, moves in ((13, 6, table, 4), (10, 2, table, 4), (10, 6, [[2, 4, 3]], 4), (10, 6, table, 3)):
        assert E.evict(w, tab, [L], [B], 4, moves, 1, 2, 1)[6] == [0]


# ------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def ra(lib_path):
    import context_ring_attention_step_gb300 as m
    m.load_library(lib_path)
    return m


def _status(ra, fn, *args):
    return getattr(ra.load_library(), fn)(*args), ra.load_library().ra_last_error().decode()


def _cache_struct(ra, pages=1 << 40, num_pages=10, page=64, heads=8, dim=128):
    from context_ring_attention_step_gb300 import kv_cache
    c = kv_cache._Cache(pages, num_pages, page, heads, dim, 0)
    _cache_struct.keep = getattr(_cache_struct, "keep", []) + [c]
    return ctypes.addressof(c)


M = 1 << 20


def test_weights_refusals(ra):
    n = ctypes.c_size_t()
    assert _status(ra, "ra_kv4_attention_workspace_bytes", 32, 8, 128, 1, ctypes.byref(n))[0] == 0
    need = n.value

    def call(c=_cache_struct(ra), q=M, qs=4096, T=4, Hq=32, table=2 * M, W=8, stride=9, lens=3 * M, cu=4 * M, R=4,
             longest=1, causal=1, scale=0.0, lse=5 * M, new=6 * M, weights=7 * M, ws=8 * M, nb=need):
        return _status(ra, "ra_kv4_weights", c, q, qs, T, Hq, table, W, stride, lens, cu, R, longest, causal, scale, lse,
                       new, weights, ws, nb, None)
    bad = lambda **kw: call(**kw)[0]
    assert bad(c=None) == 1 and bad(T=-1) == 1 and bad(R=-1) == 1 and bad(Hq=12) == 1 and bad(longest=0) == 1
    assert bad(c=_cache_struct(ra, page=48)) == 2 and bad(c=_cache_struct(ra, dim=96)) == 2
    assert bad(W=0) == 1 and bad(stride=7) == 1 and bad(scale=math.inf) == 1 and bad(scale=math.nan) == 1
    assert bad(ws=0) == 4 and bad(nb=need - 1) == 4 and bad(ws=8 * M + 16) == 4
    for name in ("q", "lse", "table", "lens", "cu", "weights"):
        assert bad(**{name: 0}) == 1, name
        assert bad(**{name: 7 * M + 3 * (1 << 16) + 2}) == 1, name
    assert bad(new=6 * M + 2) == 1 and bad(q=M + 8) == 1 and bad(qs=4095) == 1 and bad(qs=4100) == 1
    assert bad(T=(1 << 25) + 1) == 1
    # the sums are written while the rest is read; the last bytes of each count
    for at in (M + 3 * 8192 + 8188, M - 2560 + 4, 2 * M + (3 * 9 + 8) * 4 - 4, 3 * M + 12, 4 * M + 16, 5 * M + 4 * 32 * 4 - 4,
               6 * M, 8 * M + need - 4, (1 << 40) - 4):
        code, text = call(weights=at)
        assert code == 1 and "weights lie over" in text, at


def test_evict_refusals(ra):
    n = ctypes.c_size_t()
    size = lambda R: _status(ra, "ra_kv4_evict_workspace_bytes", R, ctypes.byref(n))[0]
    assert size(0) == 1 and size(-1) == 1 and size(4097) == 1 and size(4096) == 0
    assert _status(ra, "ra_kv4_evict_workspace_bytes", 4, None)[0] == 1
    assert size(4) == 0
    need = n.value
    names = ("weights", "table", "lens", "budgets", "free", "count", "out", "dropped", "src", "dst", "cout", "status")
    places = {name: (i + 1) * M for i, name in enumerate(names)}

    def call(N=10, page=64, W=8, stride=9, R=4, slack=3, recent=4, sinks=2, moves=50, num_free=10, ws=20 * M, nb=need, **kw):
        a = dict(places, **kw)
        return _status(ra, "ra_kv4_evict", a["weights"], N, page, a["table"], W, stride, a["lens"], R, a["budgets"], slack,
                       recent, sinks, moves, a["free"], num_free, a["count"], a["out"], a["dropped"], a["src"], a["dst"],
                       a["cout"], a["status"], ws, nb, None)
    bad = lambda **kw: call(**kw)[0]
    assert bad(R=0) == 1 and bad(R=4097) == 1 and bad(page=48) == 2 and bad(page=512) == 2
    assert bad(N=0) == 1 and bad(N=(1 << 30) + 1) == 1 and bad(W=0) == 1 and bad(stride=7) == 1
    assert bad(slack=-1) == 1 and bad(recent=-1) == 1 and bad(recent=5) == 1 and bad(sinks=-1) == 1
    assert bad(moves=0) == 1 and bad(moves=-1) == 1 and bad(num_free=0) == 1 and bad(num_free=-3) == 1
    assert bad(ws=0) == 4 and bad(ws=20 * M + 128) == 4 and bad(nb=need - 1) == 4
    for name in names:
        if name != "free":
            assert bad(**{name: 0}) == 1, name
        assert bad(**{name: places[name] + (4 if name in ("src", "dst") else 2)}) == 1, name
    list_bytes = 4 * 50 * 8
    for kw in (dict(out=places["budgets"]), dict(out=places["lens"] + 4), dict(dropped=places["lens"]),
               dict(dropped=places["out"] + 12), dict(src=places["dst"] + list_bytes - 8), dict(dst=places["weights"] + 2552),
               dict(src=places["table"] + 136), dict(cout=places["count"] - 0, count=places["count"], status=places["count"]),
               dict(status=places["dst"] + list_bytes - 4), dict(free=places["table"] + 4), dict(free=20 * M + need - 4),
               dict(cout=places["free"] + 36), dict(weights=places["src"] - 2552), dict(ws=places["src"])):
        code, text = call(**kw)
        assert code == 1 and "lies over" in text, kw


def test_move_refusals(ra):
    c = _cache_struct(ra)
    bad = lambda c=c, s=M, d=2 * M, n=5, w=3 * M: _status(ra, "ra_kv4_move", c, s, d, n, w, None)[0]
    assert bad(c=None) == 1 and bad(c=_cache_struct(ra, page=40)) == 2 and bad(n=-1) == 1 and bad(n=(1 << 31) + 1) == 1
    assert bad(s=0) == 1 and bad(d=0) == 1 and bad(s=M + 4) == 1 and bad(d=2 * M + 4) == 1 and bad(w=3 * M + 2) == 1
    assert bad(n=0, s=0, d=0, w=0) == 0                          # nothing to do
    cache_end = (1 << 40) + 10 * 64 * 8 * 144                    # 128 dims of K and of V: 72 bytes each
    assert bad(s=cache_end - 8) == 1 and bad(d=(1 << 40) - 32) == 1
    assert bad(s=3 * M + 2552) == 1 and bad(w=2 * M + 36) == 1 and bad(w=(1 << 40) - 2556) == 1


def test_python_checks(ra):
    c = ra.Kv4Cache(4, 64, 2, 128, device="cpu")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    q, w, s = torch.zeros(1, 4, 128, dtype=torch.bfloat16), torch.zeros(256), torch.zeros(3, dtype=torch.int64)
    args = (c, torch.zeros(1, 4, dtype=torch.int32), i32(1), i32(2), torch.zeros(4, 1), w)
    with pytest.raises(ValueError, match="gradient"):
        ra.kv4_weights(q.clone().requires_grad_(), *args)
    with pytest.raises(ValueError, match="shape"):
        ra.kv4_weights(q[0], *args)
    with pytest.raises(ValueError, match="GPU"):
        ra.kv4_weights(q, *args)
    with pytest.raises(ValueError, match="GPU"):
        ra.kv4_evict(w, args[1], i32(1), i32(1), 64, 5)
    with pytest.raises(ValueError, match="GPU"):
        ra.kv4_move(c, s, s)
