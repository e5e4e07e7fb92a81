"""4-bit key/value cache without a GPU: the oracle's formats, and what the calls refuse before any device work."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4 as O


# ------------------------------------------------------------------ the oracle's own pins

def test_scale_codes_are_fp16_numbers():
    bits = (np.arange(len(O.SCALES)).astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(bits, O.SCALES)
    assert O.SCALES[-1] == 10240 and len(O.SCALES) == 227


@pytest.mark.parametrize("x,want", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (9.0, 7)])
def test_element_ties_go_to_the_even_code(x, want):
    assert O.nearest(np.array([x]), O.ELEMENTS)[0] == want


def test_rounding_error_and_idempotence():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 128)) * np.exp(rng.standard_normal((64, 1)) * 3)
    x = torch.tensor(x).to(torch.bfloat16).double().numpy()
    v = O.rounded(x)
    amax = np.abs(x.reshape(64, 8, 16)).max(-1).repeat(16, axis=1).reshape(64, 128)
    # half the widest step (2 s of codes 4..6) plus the scale's own rounding (6 s is within 1/16 of amax)
    assert np.all(np.abs(v - x) <= amax * (1 / 6 * (1 + 1 / 16) + 1 / 16))
    # a bf16 number holds every value: 6 significant bits
    assert np.array_equal(torch.tensor(v).to(torch.bfloat16).double().numpy(), v)


def test_rounding_saturates_and_carries_nan():
    x = np.zeros((1, 48))
    x[0, 3] = 1e30
    x[0, 20] = np.inf
    x[0, 40] = 2.0 ** -30
    v = O.rounded(x)[0]
    assert v[3] == 61440 and np.all(v[:3] == 0)
    assert np.all(np.isnan(v[16:32])) and np.all(v[32:] == 0)


def test_borders_are_the_same_in_fp32():
    """Quotients of bf16 numbers by 6 and by scales decide the same in fp32 as in fp64."""
    m = np.arange(128, 256, dtype=np.float64)                    # every bf16 significand
    q64, q32 = m / 6, (m.astype(np.float32) / np.float32(6)).astype(np.float64)
    assert np.array_equal(O.nearest(q64, O.SCALES), O.nearest(q32, O.SCALES))
    for s in range(1, 16):
        for e in range(-3, 4):
            x = m * 2.0 ** e / 32
            a, b = x / s, (x.astype(np.float32) * (np.float32(1) / np.float32(s))).astype(np.float32)
            snapped = ((b + np.float32(768)) - np.float32(768)).astype(np.float64)
            keep = a < 6.5
            assert np.array_equal(O.nearest(a, O.ELEMENTS)[keep], O.nearest(snapped, O.ELEMENTS)[keep])


# ------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def ra(lib_path):
    import context_ring_attention_step_gb300 as m
    m.load_library(lib_path)
    return m


def _status(ra, fn, *args):
    return getattr(ra.load_library(), fn)(*args), ra.load_library().ra_last_error().decode()


@pytest.mark.parametrize("args,bad", [
    ((0, 64, 8, 128), 1), ((-1, 64, 8, 128), 1), ((1 << 31, 64, 8, 128), 1), ((4, 64, 0, 128), 1),
    ((4, 48, 8, 128), 2), ((4, 8, 8, 128), 2), ((4, 512, 8, 128), 2), ((4, 64, 8, 96), 2)])
def test_cache_geometry(ra, args, bad):
    with pytest.raises(ra.RingAttnError) as e:
        ra.Kv4Cache(*args, device="cpu")
    assert e.value.status == bad


def test_cache_bytes(ra):
    for d in (64, 128, 256):
        c = ra.Kv4Cache(5, 32, 3, d, device="cpu")
        assert c.pages.shape == (5, 2 * 3 * 18 * d)               # 4.5 bits an element of K and V
        assert c.pages.numel() * 8 == 2 * 5 * 32 * 3 * d * 4.5


def _cache_struct(ra, pages=4096, num_pages=4, page=64, heads=2, dim=128):
    from context_ring_attention_step_gb300.kv_cache import _Cache
    return ctypes.byref(_Cache(pages, num_pages, page, heads, dim, 0))


def test_store_and_load_refusals(ra):
    ok = _cache_struct(ra)
    store = lambda c=ok, k=4096, ks=256, v=4096, vs=256, s=4096, T=3: _status(ra, "ra_kv4_store", c, k, ks, v, vs, s, T, None)[0]
    assert store(c=None) == 1 and store(c=_cache_struct(ra, pages=0)) == 1 and store(c=_cache_struct(ra, pages=4104)) == 1
    assert store(k=0) == 1 and store(v=0) == 1 and store(s=0) == 1 and store(T=-1) == 1
    assert store(k=4104) == 1 and store(s=4100) == 1
    assert store(ks=248) == 1 and store(vs=260) == 1
    assert store(c=_cache_struct(ra, page=24)) == 2
    assert store(T=0, k=0, v=0, s=0) == 0
    load = lambda c=ok, s=4096, T=3, k=4096, v=4096: _status(ra, "ra_kv4_load", c, s, T, k, v, None)[0]
    assert load(c=None) == 1 and load(k=0) == 1 and load(v=4098) == 1 and load(s=0) == 1 and load(T=-5) == 1
    assert load(T=0, k=0, v=0, s=0) == 0


def test_tables_refusals(ra):
    def call(lens=64, new=64, R=4, table=64, W=8, stride=8, page=64, free=64, N=10, count=64, slots=16, out=128, cu=64,
             smap=64, pos=64, cout=64, status=64):
        return _status(ra, "ra_kv4_tables", lens, new, R, table, W, stride, page, free, N, count, slots, out, cu, smap,
                       pos, cout, status, None)[0]
    assert call(R=0) == 1 and call(R=4097) == 1 and call(page=100) == 2 and call(W=0) == 1 and call(stride=7) == 1
    assert call(slots=-1) == 1 and call(slots=(1 << 30) + 1) == 1
    for name in ("lens", "new", "table", "out", "cu", "smap", "pos", "status", "count", "cout"):
        assert call(**{name: 0}) == 1, name
        assert call(**{name: 62}) == 1, name
    assert call(N=0) == 1 and call(new=128) == 1


def test_attention_refusals(ra):
    n = ctypes.c_size_t()
    size = lambda *a: _status(ra, "ra_kv4_attention_workspace_bytes", *a, ctypes.byref(n))[0]
    assert size(32, 8, 128, 1) == 0 and n.value > 0
    assert size(32, 0, 128, 1) == 1 and size(33, 8, 128, 1) == 1 and size(32, 8, 100, 1) == 2 and size(32, 8, 128, 0) == 1
    need = n.value

    def call(c=_cache_struct(ra, heads=8), q=4096, qs=4096, T=4, Hq=32, table=64, W=8, stride=8, lens=64, cu=64, R=4,
             longest=1, causal=1, scale=0.0, o=4096, f32=0, lse=64, ws=4096, nb=need):
        return _status(ra, "ra_kv4_attention", c, q, qs, T, Hq, table, W, stride, lens, cu, R, longest, causal, scale,
                       o, f32, lse, ws, nb, None)[0]
    assert call(c=None) == 1 and call(T=-1) == 1 and call(R=-1) == 1 and call(Hq=12) == 1 and call(longest=0) == 1
    assert call(W=0) == 1 and call(stride=4) == 1 and call(scale=math.inf) == 1 and call(scale=math.nan) == 1
    assert call(ws=0) == 4 and call(nb=need - 1) == 4 and call(ws=4096 + 16) == 4
    for name in ("q", "o", "lse", "table", "lens", "cu"):
        assert call(**{name: 0}) == 1, name
        assert call(**{name: 4098}) == 1, name
    assert call(q=4104) == 1 and call(qs=4095 * 1) == 1 and call(qs=4100) == 1
    assert call(T=(1 << 25) + 1) == 1 and call(T=2 ** 31 - 1) == 1


def test_python_checks(ra):
    c = ra.Kv4Cache(4, 64, 2, 128, device="cpu")
    slots = torch.zeros(3, dtype=torch.int64)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ra.kv4_store(c, k, k, slots)
    with pytest.raises(ValueError, match="dtype"):
        ra.kv4_store(c, k.float(), k, slots)
    with pytest.raises(ValueError, match="GPU"):
        ra.kv4_load(c, slots)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        ra.kv4_attention(q, c, None, torch.zeros(1, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="shape"):
        ra.kv4_attention(q.detach()[0], c, None, torch.zeros(1, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="GPU"):
        ra.kv4_tables(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                      torch.zeros(2, 4, dtype=torch.int32), 64, 2)


def test_status_must_be_on_a_gpu(ra):
    with pytest.raises(ValueError, match="GPU"):
        ra.kv4_status(torch.zeros(1, dtype=torch.int32))


def test_outputs_must_not_overlap(ra):
    """Other CTAs read what one writes: refused, but for the lengths and the free count replaced in place."""
    K, M = 1 << 10, 1 << 20

    def tables(**change):
        a = dict(lens=1 * M, new=2 * M, table=3 * M, free=4 * M, count=5 * M, out=6 * M, cu=7 * M, smap=8 * M, pos=9 * M,
                 cout=10 * M, status=11 * M)
        a.update(change)
        return _status(ra, "ra_kv4_tables", a["lens"], a["new"], 4, a["table"], 8, 9, 64, a["free"], 10, a["count"], 16,
                       a["out"], a["cu"], a["smap"], a["pos"], a["cout"], a["status"], None)
    for change in (dict(out=2 * M), dict(out=1 * M + 4), dict(out=1 * M - 12), dict(cu=1 * M), dict(smap=9 * M - 8),
                   dict(pos=3 * M + 34 * 4), dict(cout=1 * M + 8), dict(cout=11 * M), dict(status=7 * M + 16),
                   dict(status=4 * M + 36), dict(free=3 * M + 24), dict(count=4 * M + 4)):
        code, text = tables(**change)
        assert code == 1 and "lies over" in text, change
    load = lambda k, v, s: _status(ra, "ra_kv4_load", _cache_struct(ra), s, 3, k, v, None)
    for k, v, s in ((M, M, K), (M, M + 3 * 512 - 16, K), (M, 2 * M, M + 8), (M, 2 * M, 2 * M + 8)):
        code, text = load(k, v, s)
        assert code == 1 and "lie over" in text
    n = ctypes.c_size_t()
    assert _status(ra, "ra_kv4_attention_workspace_bytes", 32, 8, 128, 1, ctypes.byref(n))[0] == 0

    def attention(q=M, qs=5000, o=4 * M, lse=3 * M, f32=0):
        return _status(ra, "ra_kv4_attention", _cache_struct(ra, heads=8), q, qs, 4, 32, 64, 8, 8, 64, 64, 4, 1, 1, 0.0, o,
                       f32, lse, 4096, n.value, None)
    for change in (dict(o=M), dict(o=M + 3 * 10000 + 8176), dict(o=M - 4 * 8192 + 16), dict(o=M - 4 * 8192 - 16, f32=1),
                   dict(lse=M + 16), dict(lse=4 * M + 4 * 8192 - 4), dict(lse=4 * M - 508)):
        code, text = attention(**change)
        assert code == 1 and "lie over" in text, change
