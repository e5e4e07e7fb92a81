"""Norms of queries and keys for each head, and the position rotation, in one pass.

Python side of the ``ra_qk_norm_rope_*`` calls of ``include/ring_attn.h`` (which
states the formulas and every convention).  They stand between a projection and
ring attention, or a cache step::

    rotary = Rotary(head_dim, base=500000.0)                  # once
    # training: differentiable in q, k and both weights
    q, k = qk_norm_rope(q, k, rope_positions(cu_seqlens), rotary, q_weight, k_weight)
    o, lse = ring_attention(q, k, v, cu_seqlens, cp_size)
    # generating: positions from the cache's tables (which count cached tokens: once kv4_evict has cut a
    # request, add all that it has dropped of it so far)
    q, k = qk_norm_rope_fwd(q, k, step.positions, rotary, q_weight, k_weight, out=(q, k))
    kv4_store(cache, k, v, step.slot_map)

No call synchronises; with caller-owned outputs (``out=``) and ``workspace=``
none allocates, so a step can be captured into a CUDA graph.  Calls run on the
current stream of the tensors' device.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import ring_attn as _ra
from .kv_cache import _array, _launch, _library, _on_gpu

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


# ra_norm_rope, field by field
_pack_shape = struct.Struct("=qiiiiiifiQQQQ").pack


class Rotary:
    """Frequencies of the position rotation, on the GPU.

    The first ``rotary_dim`` elements of a head (default: all; 0: none) are
    rotated in pairs (i, i + rotary_dim / 2), or (2i, 2i + 1) when
    ``interleaved``, by ``base ** (-2 i / rotary_dim)`` a position, or by
    ``inv_freq[i]`` where given (scaled frequencies for long contexts).
    """

    def __init__(self, head_dim, rotary_dim=None, base=10000.0, inv_freq=None, interleaved=False, device="cuda"):
        lib = _library()
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.interleaved = bool(interleaved)
        if not 0 <= self.rotary_dim <= self.head_dim:
            raise ValueError("rotary_dim %d outside [0, head_dim %d]" % (self.rotary_dim, self.head_dim))
        n = self.rotary_dim // 2
        freq = None
        if inv_freq is not None:
            values = [float(x) for x in (inv_freq.tolist() if hasattr(inv_freq, "tolist") else inv_freq)]
            if len(values) != n:
                raise ValueError("inv_freq has %d entries, expected rotary_dim / 2 = %d" % (len(values), n))
            freq = (ctypes.c_double * max(1, n))(*values)
        turns = (ctypes.c_uint64 * max(1, n))()
        _ra._check(lib.ra_rope_turns(self.rotary_dim, float(base), freq, turns))
        # (as int64: the same bits)
        bits = [t - (1 << 64) if t >> 63 else t for t in turns[:n]]
        self.turns = torch.tensor(bits, dtype=torch.int64).to(device)
        self.device = self.turns.device
        self.address = self.turns.data_ptr() if n else 0


def rope_positions(cu_seqlens, device="cuda"):
    """int32 [T]: every packed token's position in its document."""
    cu = [int(x) for x in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    if not cu or cu[0] != 0 or any(b < a for a, b in zip(cu, cu[1:])):
        raise ValueError("cu_seqlens must begin with 0 and not fall")
    t = torch.arange(cu[-1], dtype=_I32)
    start = torch.repeat_interleave(torch.tensor(cu[:-1], dtype=_I32),
                                    torch.tensor([b - a for a, b in zip(cu, cu[1:])], dtype=torch.int64))
    return (t - start).to(device)


def _strided(name, t, T, heads, dim, dtype, device):
    """(pointer, row stride) of a [T, heads, dim] tensor whose rows are dense.

    (One expression for the common case: a step makes several of these checks.)"""
    s = t.stride()
    if t.dtype is dtype and t.get_device() == device.index and t.shape == (T, heads, dim) and s[2] == 1 and s[1] == dim:
        return t.data_ptr(), s[0] if T > 1 else heads * dim
    if t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.shape != (T, heads, dim):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (T, heads, dim)))
    if T > 0 and (s[2] != 1 or (heads > 1 and s[1] != dim)):
        raise ValueError("%s: the heads of a row must lie one after the other (strides %s)" % (name, tuple(s)))
    return t.data_ptr(), s[0] if T > 1 else heads * dim


def _shape_of(q, k, positions, rotary, q_weight, k_weight, eps):
    """(the call's shape block, tokens, query heads, key heads, device); the shapes are checked against one another."""
    dev, D = q.device, rotary.head_dim
    if dev.type != "cuda":
        _on_gpu("q", dev)
    if q.dim() != 3 or k.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] != D or k.shape[2] != D:
        raise ValueError("q and k have shapes %s and %s, expected [T, heads, %d]" % (tuple(q.shape), tuple(k.shape), D))
    if rotary.device != dev:
        raise ValueError("rotary is on %s, expected %s" % (rotary.device, dev))
    T, Hq, _ = q.shape
    Hkv = k.shape[1]
    qw = kw = bf16 = 0
    if q_weight is not None or k_weight is not None:
        if eps is None:
            raise ValueError("q_weight and k_weight need the norm (eps)")
        wt = (k_weight if q_weight is None else q_weight).dtype
        if wt is not _F32 and wt is not _BF16:
            raise ValueError("weights have dtype %s, expected %s or %s" % (wt, _F32, _BF16))
        bf16 = wt is _BF16
        if q_weight is not None:
            qw = _array("q_weight", q_weight, (D,), wt, dev)
        if k_weight is not None:
            kw = _array("k_weight", k_weight, (D,), wt, dev)
    c = _pack_shape(T, Hq, Hkv, D, rotary.rotary_dim, rotary.interleaved, eps is not None, eps or 0.0, bf16,
                    _array("positions", positions, (T,), _I32, dev), rotary.address, qw, kw)
    return c, T, Hq, Hkv, dev


def _trained(w):
    return w is not None and w.requires_grad


def qk_norm_rope_fwd(q, k, positions, rotary, q_weight=None, k_weight=None, eps=1e-6, out=None):
    """Normed and rotated (q, k) of q [T, Hq, d] and k [T, Hkv, d] (bf16; rows may be strided).

    ``positions`` int32 [T]; a negative one makes the token's rows zero.
    ``eps=None`` leaves the norm out.  ``out=(q_out, k_out)`` writes into
    caller-owned tensors (rows may be strided); they may be q and k themselves.
    No gradient flows through it: ``qk_norm_rope`` does that.
    """
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or _trained(q_weight) or _trained(k_weight)):
        raise ValueError("qk_norm_rope_fwd has no gradient: call qk_norm_rope, or this under torch.no_grad()")
    if _ra.has_tangent(q, k, q_weight, k_weight):
        raise ValueError("qk_norm_rope_fwd has no forward-mode derivative: call it on tensors without tangents")
    c, T, Hq, Hkv, dev = _shape_of(q, k, positions, rotary, q_weight, k_weight, eps)
    D = rotary.head_dim
    qp, qs = _strided("q", q, T, Hq, D, _BF16, dev)
    kp, ks = _strided("k", k, T, Hkv, D, _BF16, dev)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=_BF16, device=dev), torch.empty((T, Hkv, D), dtype=_BF16, device=dev)
    qo, ko = out
    qop, qos = _strided("q_out", qo, T, Hq, D, _BF16, dev)
    kop, kos = _strided("k_out", ko, T, Hkv, D, _BF16, dev)
    _launch(dev, _library().ra_qk_norm_rope_fwd, c, qp, qs, kp, ks, qop, qos, kop, kos)
    return qo, ko


def qk_norm_rope_workspace(head_dim, device="cuda"):
    """Workspace for ``qk_norm_rope_bwd`` calls that take weight gradients.  Calls that may overlap need one each."""
    lib = _library()
    n = ctypes.c_size_t()
    _ra._check(lib.ra_qk_norm_rope_workspace_bytes(int(head_dim), ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def qk_norm_rope_bwd(q, k, gq, gk, positions, rotary, q_weight=None, k_weight=None, eps=1e-6, workspace=None, out=None,
                     weight_grads=True):
    """Gradients (dq, dk, dq_weight, dk_weight) from gq, gk, those of ``qk_norm_rope_fwd``'s results.

    ``gq``, ``gk``: both bf16 or both fp32, rows may be strided.  dq, dk are bf16
    (``out=(dq, dk)``: caller-owned, rows may be strided, e.g. slices of a fused
    projection's gradient); the weights' are fp32 [d], None where there is no
    weight or ``weight_grads`` is false (``out=(dq, dk, dq_weight, dk_weight)``:
    caller-owned too, None for those that are not).  No gradient flows through it, and q, k, gq and
    gk that would need one are refused (the weights may be parameters).
    """
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or gq.requires_grad or gk.requires_grad):
        raise ValueError("qk_norm_rope_bwd has no gradient: call it under torch.no_grad()")
    if _ra.has_tangent(q, k, gq, gk, q_weight, k_weight):
        raise ValueError("qk_norm_rope_bwd has no forward-mode derivative: call it on tensors without tangents")
    c, T, Hq, Hkv, dev = _shape_of(q, k, positions, rotary, q_weight, k_weight, eps)
    D = rotary.head_dim
    qp, qs = _strided("q", q, T, Hq, D, _BF16, dev)
    kp, ks = _strided("k", k, T, Hkv, D, _BF16, dev)
    gt = gq.dtype
    if gt is not _BF16 and gt is not _F32:
        raise ValueError("gq has dtype %s, expected %s or %s" % (gt, _BF16, _F32))
    gqp, gqs = _strided("gq", gq, T, Hq, D, gt, dev)
    gkp, gks = _strided("gk", gk, T, Hkv, D, gt, dev)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=_BF16, device=dev), torch.empty((T, Hkv, D), dtype=_BF16, device=dev)
    dq, dk, dqw, dkw = out if len(out) == 4 else (*out, None, None)
    dqp, dqs = _strided("dq", dq, T, Hq, D, _BF16, dev)
    dkp, dks = _strided("dk", dk, T, Hkv, D, _BF16, dev)
    if (dqw is not None and (q_weight is None or not weight_grads)) or (
            dkw is not None and (k_weight is None or not weight_grads)):
        raise ValueError("out holds the gradient of a weight that is not there or not asked for")
    dqwp = dkwp = ws = ws_bytes = 0
    if weight_grads and not (q_weight is None and k_weight is None):
        if dqw is not None:
            dqwp = _array("dq_weight", dqw, (D,), _F32, dev)
        elif q_weight is not None:
            dqw = torch.empty(D, dtype=_F32, device=dev)
            dqwp = dqw.data_ptr()
        if dkw is not None:
            dkwp = _array("dk_weight", dkw, (D,), _F32, dev)
        elif k_weight is not None:
            dkw = torch.empty(D, dtype=_F32, device=dev)
            dkwp = dkw.data_ptr()
        if workspace is None:
            workspace = qk_norm_rope_workspace(D, dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % dev)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch(dev, _library().ra_qk_norm_rope_bwd, c, qp, qs, kp, ks, gqp, gqs, gkp, gks, gt is _F32, dqp, dqs, dkp, dks,
            dqwp, dkwp, ws, ws_bytes)
    return dq, dk, dqw, dkw


class QkNormRope(torch.autograd.Function):
    """Autograd wrapper: saves the inputs and runs qk_norm_rope_bwd.  Use ``qk_norm_rope(...)``.

    The kernels' gradients are constants to autograd, so a second derivative is an error."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, rotary, eps):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions)
        ctx.rotary, ctx.eps = rotary, eps
        return qk_norm_rope_fwd(q, k, positions, rotary, q_weight, k_weight, eps)

    @staticmethod
    def backward(ctx, gq, gk):
        q, k, q_weight, k_weight, positions = ctx.saved_tensors
        need = ctx.needs_input_grad
        with torch.no_grad():
            dq, dk, dqw, dkw = qk_norm_rope_bwd(q, k, gq.contiguous(), gk.contiguous(), positions, ctx.rotary, q_weight,
                                                k_weight, ctx.eps, weight_grads=need[2] or need[3])
            cast = lambda g, w, n: g.to(w.dtype) if n and g is not None else None  # noqa: E731
            grads = (dq if need[0] else None, dk if need[1] else None, cast(dqw, q_weight, need[2]),
                     cast(dkw, k_weight, need[3]))
        return _ra.first_order("qk_norm_rope", grads, gq, gk, q, k, q_weight, k_weight) + (None, None, None)


def qk_norm_rope(q, k, positions, rotary, q_weight=None, k_weight=None, eps=1e-6):
    """Differentiable ``qk_norm_rope_fwd``: gradients flow to q, k and the weights.

    A backward pass that is captured into a CUDA graph needs leaves of its own, or that
    every graph that was recorded eagerly from the same leaves is gone by then: PyTorch adds a
    leaf's gradients up on the stream of its first graph, and a capture must not wait for that one.
    """
    return QkNormRope.apply(q, k, q_weight, k_weight, positions, rotary, eps)
