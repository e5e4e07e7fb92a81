"""Norms with rotation without a GPU: the oracle's own pins, the frequencies' table, and what the calls refuse."""

import ctypes
import sys

import numpy as np
import pytest
import torch

from oracle import rope as O


@pytest.fixture(scope="module")
def ra(lib_path):
    import context_ring_attention_step_gb300 as m
    m.load_library(lib_path)
    return m


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("rot,inter,norm", [(8, False, True), (8, True, True), (4, False, False), (0, True, True)])
def test_oracle_gradient_matches_differences(rot, inter, norm):
    rng = np.random.default_rng(5)
    T, H, d = 3, 2, 8
    x, g, w = rng.standard_normal((T, H, d)), rng.standard_normal((T, H, d)), 1 + 0.3 * rng.standard_normal(d)
    pos, f = np.array([0, 7, 100000]), O.frequencies(rot, 100.0) if rot else np.zeros(0)
    eps = 1e-3 if norm else None
    dx, dw = O.backward(x, g, pos, f, inter, w if norm else None, eps)
    loss = lambda x, w: (O.forward(x, pos, f, inter, w if norm else None, eps) * g).sum()  # noqa: E731
    h = 1e-6
    for i in np.ndindex(T, H, d):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in range(d):
            e = np.zeros(d)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_oracle_rotation_keeps_relative_positions():
    """Products of rotated rows depend on the distance of their positions only, in both layouts."""
    rng = np.random.default_rng(6)
    q, k, f = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16)), O.frequencies(16, 50.0)
    for inter in (False, True):
        dots = [(O.rotated(q, [p], f, inter) * O.rotated(k, [p - 5], f, inter)).sum() for p in (5, 12, 9000)]
        assert np.allclose(dots, dots[0], rtol=0, atol=1e-9)


# ------------------------------------------------------------------ frequencies

@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e6)])
def test_turns_hold_the_angles_at_far_positions(ra, rot, base):
    turns = [t % (1 << 64) for t in ra.Rotary(256, rot, base=base, device="cpu").turns.tolist()]
    for p in (1, 4097, 1 << 20, (1 << 31) - 1):
        got = np.array([(t * p % (1 << 64)) / 2.0 ** 64 for t in turns])
        f = O.frequencies(rot, base).astype(np.longdouble) / (2 * np.longdouble(np.pi))
        want = (f * p) % 1
        off = np.abs((got - want.astype(np.float64) + 0.5) % 1 - 0.5)
        # the frequency is a double's 53 bits of at most a turn, times the position
        assert off.max() <= 2.0 ** -53 * p + 2.0 ** -50


def test_turns_of_given_frequencies(ra):
    r = ra.Rotary(64, 8, inv_freq=[0.0, 1.0, -1.0, 0.25], device="cpu")
    t = np.array([x % (1 << 64) for x in r.turns.tolist()]) / 2.0 ** 64
    assert np.allclose(t, [0, 1 / (2 * np.pi), 1 - 1 / (2 * np.pi), 0.25 / (2 * np.pi)], rtol=0, atol=1e-15)


@pytest.mark.parametrize("kw", [dict(rotary_dim=66), dict(rotary_dim=7), dict(rotary_dim=-2), dict(base=0.0),
                                dict(base=float("inf")), dict(inv_freq=[1.0]), dict(rotary_dim=2, inv_freq=[7.0]),
                                dict(rotary_dim=2, inv_freq=[float("nan")])])
def test_rotary_refusals(ra, kw):
    with pytest.raises((ValueError, ra.RingAttnError)):
        ra.Rotary(64, device="cpu", **kw)


def test_positions_of_documents(ra):
    assert ra.rope_positions([0, 3, 3, 5], "cpu").tolist() == [0, 1, 2, 0, 1]
    assert ra.rope_positions(torch.tensor([0]), "cpu").tolist() == []
    for bad in ([], [1, 2], [0, 3, 2]):
        with pytest.raises(ValueError):
            ra.rope_positions(bad, "cpu")


def test_rows_on_the_cpu_are_refused(ra):
    rotary = ra.Rotary(64, device="cpu")
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected a GPU"):
        ra.qk_norm_rope_fwd(x, x, torch.zeros(2, dtype=torch.int32), rotary)


# ------------------------------------------------------------------ the C calls' checks (no device work before them)

A = 1 << 40          # addresses that are never touched
ROWS = 4


class _Shape(ctypes.Structure):
    """ra_norm_rope as the header has it."""

    _fields_ = [("num_tokens", ctypes.c_int64), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("weights_bf16", ctypes.c_int32),
                ("positions", ctypes.c_void_p), ("turns", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]


def shape_block(ra, **kw):
    v = dict(num_tokens=ROWS, num_q_heads=2, num_kv_heads=1, head_dim=64, rotary_dim=64, interleaved=0, norm=1, eps=1e-6,
             weights_bf16=0, positions=A + (9 << 20), turns=A + (10 << 20), q_weight=A + (11 << 20),
             k_weight=A + (12 << 20))
    v.update(kw)
    return _Shape(*[v[n] for n, _ in _Shape._fields_])


def test_the_packed_shape_is_the_structure(ra):
    from context_ring_attention_step_gb300.rope import _pack_shape
    values = (7, 6, 5, 64, 32, 1, 1, 0.5, 1, 11, 22, 33, 44)
    assert _pack_shape(*values) == bytes(_Shape(*values))


def fwd_args(**kw):
    v = dict(q=A, qs=128, k=A + (1 << 20), ks=64, qo=A + (2 << 20), qos=128, ko=A + (3 << 20), kos=64)
    v.update(kw)
    return list(v.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(head_dim=80), 2, "head_dim"), (dict(num_tokens=-1), 1, "num_tokens"), (dict(num_tokens=1 << 31), 1, "num_tokens"),
    (dict(num_q_heads=0), 1, "num_q_heads"), (dict(num_kv_heads=70000), 1, "num_kv_heads"),
    (dict(rotary_dim=20), 2, "rotary_dim"), (dict(rotary_dim=33, interleaved=1), 2, "rotary_dim"),
    (dict(rotary_dim=128), 2, "rotary_dim"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(norm=0), 1, "weights need the norm"), (dict(positions=None), 1, "positions"), (dict(turns=None), 1, "turns"),
    (dict(positions=A + 2), 1, "aligned"), (dict(q_weight=A + 2), 1, "aligned")])
def test_shape_refusals(ra, kw, status, word):
    lib = ra.load_library()
    c = shape_block(ra, **kw)
    assert lib.ra_qk_norm_rope_fwd(ctypes.addressof(c), *fwd_args(), None) == status
    assert word in lib.ra_last_error().decode()


@pytest.mark.parametrize("kw,word", [
    (dict(q=None), "q is NULL"), (dict(k=A + 8), "aligned"), (dict(qs=100), "stride"), (dict(qs=64), "stride"),
    (dict(ks=68), "stride"), (dict(qo=A + 16), "lies over"), (dict(qo=A, qos=256), "lies over"),
    (dict(ko=A), "lies over"), (dict(ko=A + (2 << 20)), "lies over"), (dict(qo=A + (9 << 20)), "lies over"),
    (dict(ko=A + (12 << 20) - 64), "lies over")])
def test_row_refusals(ra, kw, word):
    lib = ra.load_library()
    c = shape_block(ra)
    assert lib.ra_qk_norm_rope_fwd(ctypes.addressof(c), *fwd_args(**kw), None) == 1
    assert word in lib.ra_last_error().decode()


def test_backward_refusals(ra):
    lib = ra.load_library()
    n = ctypes.c_size_t()
    assert lib.ra_qk_norm_rope_workspace_bytes(64, ctypes.byref(n)) == 0
    assert lib.ra_qk_norm_rope_workspace_bytes(65, ctypes.byref(n)) == 2
    lib.ra_qk_norm_rope_workspace_bytes(64, ctypes.byref(n))
    base = dict(q=A, qs=128, k=A + (1 << 20), ks=64, gq=A + (2 << 20), gqs=128, gk=A + (3 << 20), gks=64, f=0,
                dq=A + (4 << 20), dqs=128, dk=A + (5 << 20), dks=64, dqw=A + (6 << 20), dkw=A + (7 << 20),
                ws=A + (8 << 24), wb=n.value)

    def call(shape={}, **kw):
        c = shape_block(ra, **shape)
        v = dict(base, **kw)
        return lib.ra_qk_norm_rope_bwd(ctypes.addressof(c), *v.values(), None), lib.ra_last_error().decode()

    for kw, status, word in ((dict(wb=n.value - 1), 4, "workspace"), (dict(ws=None), 4, "workspace"),
                             (dict(ws=(A + (8 << 24)) + 16), 4, "workspace"), (dict(dqw=A + (6 << 20) + 2), 1, "aligned"),
                             (dict(dq=A), 1, "lies over"), (dict(dk=A + (3 << 20)), 1, "lies over"),
                             (dict(dqw=A + (7 << 20)), 1, "lies over"), (dict(dkw=A + (8 << 24)), 1, "lies over"),
                             (dict(dqw=A + (11 << 20)), 1, "lies over"), (dict(gq=None), 1, "gq is NULL"),
                             (dict(gqs=130, f=1), 1, "stride"), (dict(ws=A), 1, "lies over")):
        got, text = call(**kw)
        assert got == status and word in text, (kw, got, text)
    got, text = call(shape=dict(q_weight=None))
    assert got == 1 and "needs the weight" in text


def test_slices_of_one_tensor_lie_beside_one_another(ra):
    """Rows of a fused tensor interleave without sharing bytes: that alone is no refusal (an unaligned turns is, first)."""
    lib = ra.load_library()
    c = shape_block(ra)
    row = 4 * 64                                                 # q (2 heads), k, and one more head
    ok = fwd_args(q=A, qs=row, k=A + 2 * 128, ks=row, qo=A, qos=row, ko=A + 3 * 128, kos=row)
    bad = fwd_args(q=A, qs=row, k=A + 2 * 128, ks=row, qo=A, qos=row, ko=A + 2 * 128 - 16, kos=row)
    assert lib.ra_qk_norm_rope_fwd(ctypes.addressof(c), *bad, None) == 1
    assert "lies over" in lib.ra_last_error().decode()
    if not torch.cuda.is_available():                            # past every check: the device is missing
        assert lib.ra_qk_norm_rope_fwd(ctypes.addressof(c), *ok, None) == 3


@pytest.mark.parametrize("which", range(4))
def test_a_lost_gradient_is_refused(ra, which):
    rotary = ra.Rotary(64, device="cpu")
    t = [torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.ones(64), torch.ones(64)]
    t[which].requires_grad_()
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="gradient"):
        ra.qk_norm_rope_fwd(t[0], t[1], pos, rotary, t[2], t[3])
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        ra.qk_norm_rope_fwd(t[0], t[1], pos, rotary, t[2], t[3])


# ------------------------------------------------------------------ second derivatives

def _stand_ins(ra, monkeypatch):
    """y = x^2 on the CPU in place of the two kernels; the weights count for nothing."""
    mod = sys.modules[ra.QkNormRope.__module__]
    monkeypatch.setattr(mod, "qk_norm_rope_fwd", lambda q, k, *a, **kw: (q * q, k * k))
    monkeypatch.setattr(mod, "qk_norm_rope_bwd",
                        lambda q, k, gq, gk, *a, **kw: ((2 * q * gq).detach(), (2 * k * gk).detach(), None, None))


@pytest.mark.parametrize("linear", [False, True])
def test_a_second_derivative_is_an_error(ra, monkeypatch, linear):
    """Kernels' gradients are constants to autograd: what would lose the rest of a second derivative raises,
    behind a loss that is linear in the results (their gradients are constants) too."""
    _stand_ins(ra, monkeypatch)
    q, k = (torch.full((2, 1, 64), v, requires_grad=True) for v in (1.5, 2.0))
    y, z = ra.qk_norm_rope(q, k, torch.zeros(2, dtype=torch.int32), None)
    loss = y.sum() + z.sum() if linear else (y * q).sum() + (z * k).sum()
    grads = torch.autograd.grad(loss, (q, k), create_graph=True)
    for g, x in zip(grads, (q, k)):
        assert torch.equal(g, (2 if linear else 3 * x) * x)
        with pytest.raises(RuntimeError, match="qk_norm_rope has no second derivative"):
            torch.autograd.grad((g * g).sum() + (x * x).sum(), x, retain_graph=True)


def test_gradients_of_frozen_inputs(ra, monkeypatch):
    """With create_graph and without: the first derivative is the same, beside inputs that need none."""
    _stand_ins(ra, monkeypatch)
    for create in (False, True):
        q, k = torch.full((2, 1, 64), 1.5, requires_grad=True), torch.full((2, 1, 64), 2.0)
        w = torch.ones(64, requires_grad=True)
        y, z = ra.qk_norm_rope(q, k, torch.zeros(2, dtype=torch.int32), None, w, None)
        dq, = torch.autograd.grad(y.sum(), q, create_graph=create)
        assert torch.equal(dq, 2 * q) and dq.requires_grad is create


@pytest.mark.parametrize("which", range(4))
def test_a_lost_gradient_of_the_gradients_is_refused(ra, which):
    rotary, pos = ra.Rotary(64, device="cpu"), torch.zeros(2, dtype=torch.int32)
    t = [torch.zeros(2, 1, 64, dtype=torch.bfloat16) for _ in range(4)]
    w = torch.ones(64, requires_grad=True)                       # (a parameter as it is)
    t[which].requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        ra.qk_norm_rope_bwd(*t, pos, rotary, w, w)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        ra.qk_norm_rope_bwd(*t, pos, rotary, w, w)
    t[which] = t[which].detach()
    with pytest.raises(ValueError, match="GPU"):
        ra.qk_norm_rope_bwd(*t, pos, rotary, w, w)


def test_a_lost_tangent_is_refused(ra, monkeypatch):
    """Forward-mode differentiation: tensors with a tangent need no gradient, and the kernels would drop it."""
    from torch.autograd import forward_ad
    rotary, pos = ra.Rotary(64, device="cpu"), torch.zeros(2, dtype=torch.int32)
    x, w = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.ones(64)
    cache, i32 = ra.Kv4Cache(4, 64, 1, 64, device="cpu"), lambda n: torch.zeros(n, dtype=torch.int32)
    tables, lse, sums = (torch.zeros(1, 4, dtype=torch.int32), i32(1), i32(2)), torch.zeros(1, 2), torch.zeros(256)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="GPU"):             # no tangent: on to the other checks
            ra.qk_norm_rope_fwd(x, x, pos, rotary, w, w)
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call, args, at in ((ra.qk_norm_rope_fwd, (x, x, pos, rotary, w, w), (0, 1, 4, 5)),
                               (ra.qk_norm_rope_bwd, (x, x, x, x, pos, rotary, w, w), (0, 1, 2, 3, 6, 7)),
                               (ra.kv4_attention, (x, cache) + tables, (0,)),
                               (ra.kv4_weights, (x, cache) + tables + (lse, sums), (0, 5, 6))):
            for i in at:
                with pytest.raises(ValueError, match="forward-mode"):
                    call(*[dual(a) if j == i else a for j, a in enumerate(args)])
        _stand_ins(ra, monkeypatch)
        with pytest.raises(RuntimeError):                        # the differentiable call has no rule for it
            ra.qk_norm_rope(dual(x), x, pos, None)
