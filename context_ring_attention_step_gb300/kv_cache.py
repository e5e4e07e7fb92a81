"""Key/value cache held in 4 bits: pages, store, load and attention over it.

Python side of the ``ra_kv4_*`` calls of ``include/ring_attn.h`` (which states
the format, the page layout and every convention).  A serving loop next to
ring attention uses them like this::

    cache = Kv4Cache(num_pages, 64, num_kv_heads, head_dim)      # one per layer
    # a prompt: its attention by ring_attn_fwd, its keys and values into the cache
    step = kv4_tables(lens, new_lens, table, 64, num_slots, free_pages, free_count)
    kv4_store(cache, k, v, step.slot_map)
    # then token by token (or a few tokens, or the next part of a prompt)
    step = kv4_tables(step.kv_lens, ones, table, 64, batch, free_pages, step.free_count)
    kv4_store(cache, k1, v1, step.slot_map)
    o, lse = kv4_attention(q1, cache, table, step.kv_lens, step.cu_new, max_q_len=1)

and, to keep every request within a budget, the attention weight that its
tokens receive in the step, and once in a while the lightest ones' removal::

    kv4_weights(q1, cache, table, step.kv_lens, step.cu_new, lse, sums, new_lens=ones, max_q_len=1)
    cut = kv4_evict(sums, table, step.kv_lens, budgets, 64, max_moves, slack, recent, sinks, free_pages, step.free_count)
    kv4_move(cache, cut.src_slots, cut.dst_slots, weights=sums)      # before the next kv4_store
    # cut.kv_lens and cut.free_count go into the next kv4_tables; positions: its own + all cut.dropped so far

No call synchronises unless ``check=True``, and with caller-owned outputs
(``out=``) and ``workspace=`` none allocates, so a step can be captured into a
CUDA graph.  Calls run on the current stream of the tensors' device.
"""

from __future__ import annotations

import collections
import ctypes

import torch

from . import ring_attn as _ra

_current_raw_stream = torch._C._cuda_getCurrentRawStream


class _Cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Kv4Cache:
    """Pages of one layer's keys and values in 4 bits (4.5 with the scales).

    ``pages`` is a uint8 tensor [num_pages, bytes of a page]; its content is
    written by ``kv4_store`` only.
    """

    def __init__(self, num_pages, page_size, num_kv_heads, head_dim, device="cuda"):
        lib = _ra.load_library()
        n = ctypes.c_size_t()
        _ra._check(lib.ra_kv4_cache_bytes(int(num_pages), int(page_size), int(num_kv_heads), int(head_dim),
                                          ctypes.byref(n)))
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.num_kv_heads, self.head_dim = int(num_kv_heads), int(head_dim)
        self.pages = torch.zeros(self.num_pages, n.value // self.num_pages, dtype=torch.uint8, device=device)
        self.device = self.pages.device
        self._c = _Cache(self.pages.data_ptr(), self.num_pages, self.page_size, self.num_kv_heads, self.head_dim, 0)
        self._ref = ctypes.addressof(self._c)


Kv4Tables = collections.namedtuple("Kv4Tables", "kv_lens cu_new slot_map positions free_count status")


_I32, _I64, _BF16, _F32 = torch.int32, torch.int64, torch.bfloat16, torch.float32
_current_device = torch._C._cuda_getDevice


def _library():
    return _ra._lib or _ra.load_library()


def _launch(device, fn, *args):
    """fn(*args, stream) on the device's current stream, with the device current."""
    i = device.index
    if _current_device() == i:
        status = fn(*args, _current_raw_stream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, _current_raw_stream(i))
    if status:
        _ra._check(status)


def _on_gpu(name, device):
    if device.type != "cuda":
        raise ValueError("%s is on %s, expected a GPU" % (name, device))


def _array(name, t, shape, dtype, device):
    """Pointer of a contiguous tensor with exactly this shape, type and device.

    (One expression for the common case: a step makes a dozen of these checks,
    and they are most of its host time.)"""
    if t.dtype is dtype and t.get_device() == device.index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    raise ValueError("%s must be contiguous" % name)


def _rows(name, t, heads, dim, device):
    """(pointer, row stride) of a [T, heads, dim] bf16 tensor whose rows are dense."""
    if t.dtype is not _BF16:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, _BF16))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError("%s has shape %s, expected [T, %d, %d]" % (name, tuple(shape), heads, dim))
    if shape[0] == 0:
        return 0, heads * dim
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != dim):
        raise ValueError("%s: the heads of a row must lie one after the other (strides %s)" % (name, tuple(s)))
    return t.data_ptr(), s[0] if shape[0] > 1 else heads * dim


def _table(block_table, num_requests, device):
    """(pointer, width, row stride) of an int32 [num_requests, width] tensor whose rows are dense."""
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != num_requests:
        raise ValueError("block_table has shape %s, expected [%d, pages]" % (tuple(shape), num_requests))
    if block_table.dtype is not _I32 or block_table.device != device:
        raise ValueError("block_table must be an int32 tensor on %s" % device)
    w = shape[1]
    s = block_table.stride()
    if w > 1 and s[1] != 1:
        raise ValueError("block_table rows must be dense")
    return block_table.data_ptr(), w, s[0] if num_requests > 1 else max(w, 1)


def kv4_tables_out(num_requests, num_slots, device="cuda"):
    """Caller-owned outputs for ``kv4_tables(out=...)``."""
    i32 = dict(dtype=torch.int32, device=device)
    return Kv4Tables(torch.empty(num_requests, **i32), torch.empty(num_requests + 1, **i32),
                     torch.empty(num_slots, dtype=torch.int64, device=device), torch.empty(num_slots, **i32),
                     torch.empty(1, **i32), torch.empty(1, **i32))


def kv4_tables(kv_lens, new_lens, block_table, page_size, num_slots, free_pages=None, free_count=None, out=None,
               check=False):
    """One step's page bookkeeping (ra_kv4_tables): returns a ``Kv4Tables``.

    ``kv_lens`` [R] and ``new_lens`` [R] (int32): tokens cached before the step
    and tokens it adds, -1 for a request that leaves.  ``block_table`` [R, W] and
    ``free_pages`` [N] are updated in place; ``free_pages=None`` only maps (the
    block table already holds the pages; the free count is handed on, 0 if there is
    none).  ``num_slots``: length of the slot map (-1 behind the last new token).
    ``out`` may name ``kv_lens`` and ``free_count`` themselves as outputs.  A step
    that cannot be done (not enough pages, ...) changes nothing and says so in
    ``status``; a step over pages that are none (negative) is made, and its status
    says that.  ``check=True`` synchronises and raises.
    """
    lib = _library()
    dev, R = kv_lens.device, kv_lens.shape[0]
    _on_gpu("kv_lens", dev)
    num_slots = int(num_slots)
    if out is None:
        out = kv4_tables_out(R, num_slots, dev)
    per_r, one = (R,), (1,)
    lens = _array("kv_lens", kv_lens, per_r, _I32, dev)
    new = _array("new_lens", new_lens, per_r, _I32, dev)
    table, width, stride = _table(block_table, R, dev)
    free = count = None
    num_pages = 0
    if free_pages is not None:
        if free_count is None:
            raise ValueError("free_pages needs free_count")
        num_pages = free_pages.shape[0]
        free = _array("free_pages", free_pages, (num_pages,), _I32, dev)
    if free_count is not None:
        count = _array("free_count", free_count, one, _I32, dev)
    o_lens, o_cu, o_slots, o_pos, o_count, o_status = out
    _launch(dev, lib.ra_kv4_tables, lens, new, R, table, width, stride, int(page_size), free, num_pages, count,
            num_slots, _array("out.kv_lens", o_lens, per_r, _I32, dev),
            _array("out.cu_new", o_cu, (R + 1,), _I32, dev),
            _array("out.slot_map", o_slots, (num_slots,), _I64, dev),
            _array("out.positions", o_pos, (num_slots,), _I32, dev),
            _array("out.free_count", o_count, one, _I32, dev),
            _array("out.status", o_status, one, _I32, dev))
    if check:
        kv4_status(out.status)
    return out


def kv4_store(cache, k, v, slot_map, check=False):
    """Round rows k, v [T, num_kv_heads, head_dim] (bf16) to 4 bits into the slots of ``slot_map`` [T].

    Rows may be strided (slices of a projection's output).  Rows with a negative
    slot, or one outside the cache, are left out.  A slot must not occur twice;
    ``check=True`` synchronises and raises if one does or lies outside.
    """
    lib = _library()
    dev, T = cache.device, slot_map.shape[0]
    kp, ks = _rows("k", k, cache.num_kv_heads, cache.head_dim, dev)
    vp, vs = _rows("v", v, cache.num_kv_heads, cache.head_dim, dev)
    _on_gpu("cache", dev)
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError("k, v and slot_map have %d, %d and %d rows" % (k.shape[0], v.shape[0], T))
    slots = _array("slot_map", slot_map, (T,), _I64, dev)
    if check:
        used = slot_map[slot_map >= 0]
        if used.numel() and int(used.max()) >= cache.num_pages * cache.page_size:
            raise ValueError("slot_map has a slot outside the cache")
        if torch.unique(used).numel() != used.numel():
            raise ValueError("slot_map has a slot twice")
    _launch(dev, lib.ra_kv4_store, cache._ref, kp, ks, vp, vs, slots, T)


def kv4_load(cache, slot_map, out=None):
    """The cached rows of ``slot_map`` [T] as bf16 (k, v) [T, num_kv_heads, head_dim], exactly.

    Rows with a negative slot, or one outside the cache, become zero.
    """
    lib = _library()
    dev, T = cache.device, slot_map.shape[0]
    _on_gpu("cache", dev)
    shape = (T, cache.num_kv_heads, cache.head_dim)
    slots = _array("slot_map", slot_map, (T,), _I64, dev)
    if out is None:
        out = (torch.empty(shape, dtype=torch.bfloat16, device=dev), torch.empty(shape, dtype=torch.bfloat16, device=dev))
    k, v = out
    _launch(dev, lib.ra_kv4_load, cache._ref, slots, T, _array("k", k, shape, _BF16, dev),
            _array("v", v, shape, _BF16, dev))
    return k, v


def kv4_attention_workspace(cache, num_q_tokens, num_q_heads, max_q_len=None):
    """Workspace (zeroed, as its first use needs it) for ``kv4_attention`` calls with up to
    ``max_q_len`` query tokens a request (default: ``num_q_tokens``).  Calls that may overlap
    need one each; calls in turn may share one that is large enough for all of them."""
    lib = _ra.load_library()
    n = ctypes.c_size_t()
    longest = max(1, int(num_q_tokens if max_q_len is None else max_q_len))
    _ra._check(lib.ra_kv4_attention_workspace_bytes(int(num_q_heads), cache.num_kv_heads, cache.head_dim, longest,
                                                    ctypes.byref(n)))
    return torch.zeros(n.value, dtype=torch.uint8, device=cache.device)


def kv4_attention(q, cache, block_table, kv_lens, cu_q, causal=True, scale=None, o_fp32=False, max_q_len=None,
                  workspace=None, out=None, check=False):
    """Attention of packed query rows over the cache: returns (o [Tq, Hq, d], lse [Hq, Tq] fp32).

    Request r brings rows ``cu_q[r]:cu_q[r+1]`` of ``q`` [Tq, Hq, d] (bf16, rows
    may be strided) and has ``kv_lens[r]`` cached tokens, the rows' own among
    them (``causal``: row i of n sees keys up to ``kv_lens[r] - n + i``).
    ``max_q_len``: query tokens of the longest request.  It selects the kernels,
    so give it: the default, Tq, is right for one request, but lets a step of
    single tokens launch the kernel of long requests too (128 of them over 2000
    tokens: 75 us instead of 69) and makes the default workspace a large one.
    ``scale`` <= 0 or None selects 1/sqrt(d).  Not differentiable.
    ``check=True`` synchronises and raises if the lengths, offsets or pages were
    out of range; without it, look at ``kv4_status(workspace)`` now and then: keys
    on pages outside the cache are left out of the rows silently.
    """
    lib = _library()
    if q.requires_grad and torch.is_grad_enabled():
        raise ValueError("kv4_attention has no gradient: call it under torch.no_grad()")
    if _ra.has_tangent(q):
        raise ValueError("kv4_attention has no forward-mode derivative: call it on tensors without tangents")
    dev, R = cache.device, kv_lens.shape[0]
    if q.dim() != 3:
        raise ValueError("q has shape %s, expected [T, heads, %d]" % (tuple(q.shape), cache.head_dim))
    _on_gpu("cache", dev)
    T, Hq, D = q.shape
    qp, qs = _rows("q", q, Hq, cache.head_dim, dev)
    table, width, stride = _table(block_table, R, dev)
    lens = _array("kv_lens", kv_lens, (R,), _I32, dev)
    cu = _array("cu_q", cu_q, (R + 1,), _I32, dev)
    ot = torch.float32 if o_fp32 else torch.bfloat16
    if out is None:
        o = torch.zeros((T, Hq, D), dtype=ot, device=dev)
        lse = torch.full((Hq, T), float("-inf"), dtype=torch.float32, device=dev)
    else:
        o, lse = out
    longest = max(1, int(T if max_q_len is None else max_q_len))
    if workspace is None:
        workspace = kv4_attention_workspace(cache, T, Hq, longest)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    _launch(dev, lib.ra_kv4_attention, cache._ref, qp, qs, T, Hq, table, width, stride, lens, cu, R, longest,
            int(bool(causal)), float(scale) if scale else 0.0, _array("o", o, (T, Hq, D), ot, dev), int(bool(o_fp32)),
            _array("lse", lse, (Hq, T), _F32, dev), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    if check:
        kv4_status(workspace)
    return o, lse


def kv4_weights(q, cache, block_table, kv_lens, cu_q, lse, weights, new_lens=None, causal=True, scale=None,
                max_q_len=None, workspace=None, check=False):
    """Add to ``weights`` the attention weight that every cached token receives from the query rows.

    ``q``, ``block_table``, ``kv_lens``, ``cu_q``, ``causal``, ``scale`` and
    ``max_q_len`` as for ``kv4_attention``, and ``lse`` [Hq, Tq] from it:
    ``weights[slot] += sum of exp(scale q . k - lse)`` over the rows and query
    heads that see the slot's token.  ``weights``: fp32 [num_pages * page_size],
    updated in place (and returned).  ``new_lens`` [R] (int32): the sums of a
    request's last tokens, as many as the step added, begin at zero.
    ``workspace``: as for ``kv4_attention``, one for both.  ``check=True`` synchronises
    and raises if lengths, offsets or pages were out of range.
    """
    lib = _library()
    if q.requires_grad and torch.is_grad_enabled():
        raise ValueError("kv4_weights has no gradient: call it under torch.no_grad()")
    if _ra.has_tangent(q, lse, weights):
        raise ValueError("kv4_weights has no forward-mode derivative: call it on tensors without tangents")
    dev, R = cache.device, kv_lens.shape[0]
    if q.dim() != 3:
        raise ValueError("q has shape %s, expected [T, heads, %d]" % (tuple(q.shape), cache.head_dim))
    _on_gpu("cache", dev)
    T, Hq, D = q.shape
    qp, qs = _rows("q", q, Hq, cache.head_dim, dev)
    table, width, stride = _table(block_table, R, dev)
    lens = _array("kv_lens", kv_lens, (R,), _I32, dev)
    cu = _array("cu_q", cu_q, (R + 1,), _I32, dev)
    new = None if new_lens is None else _array("new_lens", new_lens, (R,), _I32, dev)
    longest = max(1, int(T if max_q_len is None else max_q_len))
    if workspace is None:
        workspace = kv4_attention_workspace(cache, T, Hq, longest)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    _launch(dev, lib.ra_kv4_weights, cache._ref, qp, qs, T, Hq, table, width, stride, lens, cu, R,
            longest, int(bool(causal)), float(scale) if scale else 0.0,
            _array("lse", lse, (Hq, T), _F32, dev), new,
            _array("weights", weights, (cache.num_pages * cache.page_size,), _F32, dev), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    if check:
        kv4_status(workspace)
    return weights


Kv4Eviction = collections.namedtuple("Kv4Eviction", "kv_lens dropped src_slots dst_slots free_count status")


def kv4_evict_out(num_requests, max_moves, device="cuda"):
    """Caller-owned outputs for ``kv4_evict(out=...)``."""
    i32, i64 = dict(dtype=torch.int32, device=device), dict(dtype=torch.int64, device=device)
    return Kv4Eviction(torch.empty(num_requests, **i32), torch.empty(num_requests, **i32),
                       torch.empty(num_requests, max_moves, **i64), torch.empty(num_requests, max_moves, **i64),
                       torch.empty(1, **i32), torch.empty(1, **i32))


def kv4_evict_workspace(num_requests, device="cuda"):
    """Workspace (zeroed, as its first use needs it) for ``kv4_evict``.  Calls that may overlap need one each."""
    n = ctypes.c_size_t()
    _ra._check(_library().ra_kv4_evict_workspace_bytes(int(num_requests), ctypes.byref(n)))
    return torch.zeros(n.value, dtype=torch.uint8, device=device)


def kv4_evict(weights, block_table, kv_lens, budgets, page_size, max_moves, slack=0, recent=0, sinks=0, free_pages=None,
              free_count=None, workspace=None, out=None, check=False):
    """Which cached tokens go, by the sums of ``kv4_weights`` (ra_kv4_evict): returns a ``Kv4Eviction``.

    Request r with more than ``budgets[r]`` (int32 [R], negative: no budget) +
    ``slack`` tokens is cut to its budget: the first ``sinks``, the last ``recent``
    (at most ``slack`` + 1) and otherwise the tokens with the largest ``weights`` stay.
    ``src_slots`` and ``dst_slots`` [R, max_moves] name the rows that move into the
    places of dropped ones (-1 behind the last): hand them to ``kv4_move``, for every layer
    that shares the block table, before the next tokens are stored.
    ``dropped`` [R]: tokens that went (a position counts them: index + all dropped
    so far).  Pages behind the new lengths go to ``free_pages``.  ``out`` may name ``kv_lens``
    and ``free_count`` themselves as outputs.  A request that cannot be cut is left alone,
    and ``status`` says why; ``check=True`` synchronises and raises.
    """
    lib = _library()
    dev, R = kv_lens.device, kv_lens.shape[0]
    _on_gpu("kv_lens", dev)
    page_size, max_moves = int(page_size), int(max_moves)
    if out is None:
        out = kv4_evict_out(R, max_moves, dev)
    slots = weights.shape[0]
    w = _array("weights", weights, (slots,), _F32, dev)
    if page_size < 1 or slots % page_size:
        raise ValueError("weights has %d entries, not a multiple of page_size %d" % (slots, page_size))
    per_r, one, lists = (R,), (1,), (R, max_moves)
    table, width, stride = _table(block_table, R, dev)
    free = count = None
    num_free = 0
    if free_pages is not None:
        if free_count is None:
            raise ValueError("free_pages needs free_count")
        num_free = free_pages.shape[0]
        free = _array("free_pages", free_pages, (num_free,), _I32, dev)
    if free_count is not None:
        count = _array("free_count", free_count, one, _I32, dev)
    if workspace is None:
        workspace = kv4_evict_workspace(R, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    o_lens, o_dropped, o_src, o_dst, o_count, o_status = out
    _launch(dev, lib.ra_kv4_evict, w, slots // page_size, page_size, table, width, stride,
            _array("kv_lens", kv_lens, per_r, _I32, dev), R, _array("budgets", budgets, per_r, _I32, dev), int(slack),
            int(recent), int(sinks), max_moves, free, num_free, count, _array("out.kv_lens", o_lens, per_r, _I32, dev),
            _array("out.dropped", o_dropped, per_r, _I32, dev), _array("out.src_slots", o_src, lists, _I64, dev),
            _array("out.dst_slots", o_dst, lists, _I64, dev), _array("out.free_count", o_count, one, _I32, dev),
            _array("out.status", o_status, one, _I32, dev), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    if check:
        kv4_status(out.status)
    return out


def kv4_move(cache, src_slots, dst_slots, weights=None, check=False):
    """Copy cached rows, as they are, from ``src_slots`` to ``dst_slots`` (int64, of one shape).

    Pairs with a slot that is negative or outside the cache are left out.
    ``weights`` [num_pages * page_size] (fp32): the slots' sums go along.  A slot that is
    written must occur only once among all of them; ``check=True`` synchronises and
    raises if one occurs twice.
    """
    lib = _library()
    dev, n = cache.device, src_slots.numel()
    _on_gpu("cache", dev)
    src = _array("src_slots", src_slots, src_slots.shape, _I64, dev)
    dst = _array("dst_slots", dst_slots, src_slots.shape, _I64, dev)
    end = cache.num_pages * cache.page_size
    w = None if weights is None else _array("weights", weights, (end,), _F32, dev)
    if check:
        inside = lambda x: (x >= 0) & (x < end)  # noqa: E731
        pairs = inside(src_slots) & inside(dst_slots)
        written = dst_slots[pairs]
        if torch.unique(written).numel() != written.numel() or bool(torch.isin(written, src_slots[pairs]).any()):
            raise ValueError("a slot of dst_slots occurs twice, or in src_slots")
    _launch(dev, lib.ra_kv4_move, cache._ref, src, dst, n, w)


def kv4_status(status):
    """Synchronise and raise if the status word at the start of ``status`` (``Kv4Tables.status``,
    ``Kv4Eviction.status``, or the workspace of ``kv4_attention`` or ``kv4_weights``) reports a refusal."""
    lib = _library()
    _on_gpu("status", status.device)
    _launch(status.device, lib.ra_kv4_status, status.data_ptr())
