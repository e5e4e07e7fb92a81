"""Norms with rotation on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, an fp32 half step):
  * forward: the sum of squares adds 8 terms in a chain and 3 to 5 in a tree (13 u
    of it, half of that for its root), rsqrtf and the divisions 6 u, the angle
    2^-22 turns' worth of pi and sin, cos 4 u, products and the sum 6 u: less than
    2^-18 of |u_a| + |u_b|, and half a step of bf16 at the end;
  * backward: the same on r (|h w| + |n| mean |h w n|), with |h| at most |g_a| + |g_b|;
  * weights' gradients: at most 64 terms in a chain beside them (a warp's rows,
    then 8 warps, then 80 CTAs and 8): 2^-16 of the sum of magnitudes.
"""

import math

import numpy as np
import pytest
import torch

from oracle import attention as A, rope as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra(lib_path):
    import context_ring_attention_step_gb300 as m
    m.load_library(lib_path)
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


TINY = 2.0 ** -133                                               # bf16's smallest step


def case(T, Hq, Hkv, d, seed=0, fused=True, far=True, w=torch.float32):
    """q, k, v as slices of one projection's output (fused) or dense; positions, some of them none."""
    g = torch.Generator().manual_seed(1000 * T + 10 * d + Hq + seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g) * torch.exp(torch.randn(T, Hq + 2 * Hkv, 1, generator=g))
    qkv = qkv.to(torch.bfloat16).cuda()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, (1 << 31) - 1 if far else 8192, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[torch.rand(T, generator=g) < 0.1] = -1
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(w).cuda() for _ in range(2)) if w else (None, None)
    return q, k, pos.cuda(), wq, wk


def spread(x, freq, inter):
    """|x_a| + |x_b| at the elements of a pair, |x| elsewhere."""
    a, b = O.pairs(2 * len(freq), inter)
    m = np.abs(x).copy()
    m[..., a] = m[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return m


def check_fwd(got, x, pos, freq, inter, w, eps):
    x, pos, w = f64(x), pos.cpu().numpy(), None if w is None else f64(w)
    want = O.forward(x, pos, freq, inter, w, eps)
    u = x
    if eps is not None:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    tol = half_step(torch.bfloat16) * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -18 * spread(u, freq, inter) + TINY
    assert np.all(np.abs(f64(got) - want) <= tol)


def check_bwd(got, dw, x, g, pos, freq, inter, w, eps):
    x, g, pos, w = f64(x), f64(g), pos.cpu().numpy(), None if w is None else f64(w)
    want, dw_want = O.backward(x, g, pos, freq, inter, w, eps)
    h = spread(g, freq, inter)
    if eps is None:
        m = h
    else:
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        n, hw = np.abs(x * r), h * (1.0 if w is None else np.abs(w))
        m = r * (hw + n * (hw * n).mean(-1, keepdims=True))
    tol = half_step(torch.bfloat16) * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -18 * m + TINY
    assert np.all(np.abs(f64(got) - want) <= tol)
    if dw is not None:
        live = (pos >= 0)[:, None, None]
        assert np.all(np.abs(f64(dw) - dw_want) <= 2.0 ** -16 * (np.where(live, h * n, 0)).sum((0, 1)) + 1e-30)


SHAPES = [  # T, Hq, Hkv, d, rotary_dim, interleaved, norm, weights
    (1, 1, 1, 64, 64, False, True, torch.float32),
    (1, 32, 8, 128, 128, False, True, torch.bfloat16),
    (7, 3, 3, 64, 32, False, True, torch.bfloat16),
    (64, 32, 8, 128, 128, False, True, torch.float32),
    (129, 5, 1, 128, 64, True, True, torch.float32),
    (333, 7, 2, 256, 64, False, True, torch.float32),
    (33, 9, 3, 256, 256, True, True, torch.bfloat16),
    (50, 4, 2, 128, 18, True, True, None),
    (50, 4, 2, 128, 0, False, True, torch.float32),
    (77, 6, 2, 64, 64, True, False, None),
    (77, 6, 2, 128, 96, False, False, None),
    (78, 3, 2, 64, 24, False, True, torch.bfloat16),
    (5003, 4, 2, 64, 16, False, True, torch.float32),
    (4999, 17, 1, 128, 128, False, True, torch.float32),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,norm,w", SHAPES)
def test_forward_and_backward(ra, T, Hq, Hkv, d, rot, inter, norm, w):
    q, k, pos, wq, wk = case(T, Hq, Hkv, d, w=w)
    rotary = ra.Rotary(d, rot, base=10000.0, interleaved=inter)
    freq, eps = (O.frequencies(rot, 10000.0) if rot else np.zeros(0)), 1e-6 if norm else None
    qo, ko = ra.qk_norm_rope_fwd(q, k, pos, rotary, wq, wk, eps=eps)
    check_fwd(qo, q, pos, freq, inter, wq, eps)
    check_fwd(ko, k, pos, freq, inter, wk, eps)
    for gt in (torch.bfloat16, torch.float32):
        gen = torch.Generator().manual_seed(T)
        gq = torch.randn(q.shape, generator=gen).to(gt).cuda()
        gk = torch.randn(k.shape, generator=gen).to(gt).cuda()
        dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk, eps=eps)
        assert (dwq is None) == (wq is None) and (dwk is None) == (wk is None)
        check_bwd(dq, dwq, q, gq, pos, freq, inter, wq, eps)
        check_bwd(dk, dwk, k, gk, pos, freq, inter, wk, eps)


@pytest.mark.parametrize("inter", [False, True])
def test_one_weight_only(ra, inter):
    q, k, pos, wq, wk = case(40, 4, 2, 128)
    rotary, freq = ra.Rotary(128, interleaved=inter), O.frequencies(128, 10000.0)
    gq, gk = torch.ones_like(q).contiguous(), torch.ones_like(k).contiguous()
    for a, b in ((wq, None), (None, wk)):
        qo, ko = ra.qk_norm_rope_fwd(q, k, pos, rotary, a, b)
        check_fwd(qo, q, pos, freq, inter, a, 1e-6)
        check_fwd(ko, k, pos, freq, inter, b, 1e-6)
        dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, a, b)
        check_bwd(dq, dwq, q, gq, pos, freq, inter, a, 1e-6)
        check_bwd(dk, dwk, k, gk, pos, freq, inter, b, 1e-6)
        assert (dwq is None) != (dwk is None)
    assert ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk, weight_grads=False)[2:] == (None, None)


def test_gradient_matches_differences(ra):
    """The backward pass against central differences of the forward one.

    The difference's own curvature is the oracle's (fp64, the same points); what is
    left are the results' roundings, half a bf16 step of each y on both sides, over
    the step, and the backward's."""
    d, rotary, freq = 64, ra.Rotary(64, 32), O.frequencies(32, 10000.0)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 1, d, generator=g).to(torch.bfloat16)
    w = 1 + 0.3 * torch.randn(d, generator=g)
    gy = torch.randn(1, 1, d, generator=g).to(torch.bfloat16)
    pos, zero = torch.tensor([11], dtype=torch.int32), torch.zeros(2 * d, 1, d, dtype=torch.bfloat16).cuda()
    dx = f64(ra.qk_norm_rope_bwd(x.cuda(), zero[:1], gy.cuda(), zero[:1], pos.cuda(), rotary, w.cuda(), w.cuda(),
                                 eps=0.5)[0]).flatten()
    many = x.repeat(2 * d, 1, 1).float()
    many[torch.arange(d), 0, torch.arange(d)] += 0.25
    many[d + torch.arange(d), 0, torch.arange(d)] -= 0.25
    many = many.to(torch.bfloat16)
    y = f64(ra.qk_norm_rope_fwd(many.cuda(), zero, pos.expand(2 * d).contiguous().cuda(), rotary, w.cuda(), w.cuda(),
                                eps=0.5)[0])
    ref = O.forward(f64(many), pos.expand(2 * d).numpy(), freq, False, f64(w), 0.5)
    step = f64(many[:d].double() - many[d:].double()).sum((1, 2))
    slope, exact = (((t[:d] - t[d:]) * f64(gy)).sum((1, 2)) / step for t in (y, ref))
    dx_ref, _ = O.backward(f64(x), f64(gy), pos.numpy(), freq, False, f64(w), 0.5)
    rounding = ((np.abs(ref[:d]) + np.abs(ref[d:])) * np.abs(f64(gy))).sum((1, 2)) * (half_step(torch.bfloat16) + 2.0 ** -15) / step
    back = half_step(torch.bfloat16) * np.abs(dx_ref.flatten()) * (1 + 2.0 ** -7) + 2.0 ** -12
    assert np.all(np.abs(slope - dx) <= rounding + np.abs(exact - dx_ref.flatten()) + back)
    assert np.abs(exact - dx_ref.flatten()).max() < 0.1          # the curvature does not hide the gradient
    assert rounding.max() < 1.0


def test_rows_at_the_ends_of_the_number_range(ra):
    """Squares beyond fp32's range on either side, zero rows, infinities and NaN."""
    d, rotary, freq = 128, ra.Rotary(128), O.frequencies(128, 10000.0)
    g = torch.Generator().manual_seed(8)
    base = torch.randn(12, 1, d, generator=g)
    scale = torch.tensor([2.0 ** e for e in (0, 100, 120, 63, 62, -60, -70, -100, -120, -40, 110, 1)]).view(12, 1, 1)
    x = (base * scale).to(torch.bfloat16).cuda()
    pos = torch.arange(12, dtype=torch.int32).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    for eps in (1e-6, 1e-38, 0.0):
        y, _ = ra.qk_norm_rope_fwd(x, x.clone(), pos, rotary, w, w, eps=eps)
        check_fwd(y, x, pos, freq, False, w, eps)
        gy = torch.randn(12, 1, d, generator=g).to(torch.bfloat16).cuda()
        dx, _, dw, _ = ra.qk_norm_rope_bwd(x, x.clone(), gy, gy.clone(), pos, rotary, w, w, eps=eps)
        want, _ = O.backward(f64(x), f64(gy), pos.cpu().numpy(), freq, False, f64(w), eps)
        fits = np.abs(want) < 2.0 ** 126                         # (beyond: no bf16 number, or the last few)
        rows = fits.all(axis=(1, 2))
        check_bwd(dx[rows], None, x[rows], gy[rows], pos[rows], freq, False, w, eps)
    z = torch.zeros(2, 1, d, dtype=torch.bfloat16).cuda()
    z[1, 0, 5], = torch.tensor([float("inf")]).to(torch.bfloat16)
    z[1, 0, 6] = 1.0
    p = torch.tensor([3, 4], dtype=torch.int32).cuda()
    y, _ = ra.qk_norm_rope_fwd(z, z.clone(), p, rotary, w, w)
    assert torch.all(y[0] == 0)
    # 1 / sqrt(inf) = 0: the infinity becomes NaN, and its partner 5 + 64 with it; the others zero
    bad = torch.isnan(y[1, 0]).cpu()
    assert bad.nonzero().flatten().tolist() == [5, 69] and torch.all(y[1, 0].cpu()[~bad] == 0)
    z[1, 0, 6] = float("nan")
    y, _ = ra.qk_norm_rope_fwd(z, z.clone(), p, rotary, w, w)
    assert torch.isnan(y[1]).all() and not torch.isnan(y[0]).any()
    # without the norm an infinity stays where it is, beside the rotated part too
    part = ra.Rotary(d, 64)
    y, _ = ra.qk_norm_rope_fwd(z[:1].clone().index_fill_(2, torch.tensor([100]).cuda(), float("inf")), z[:1], p[:1], part,
                               eps=None)
    assert torch.isinf(y[0, 0, 100]) and torch.isfinite(y[0, 0, :100]).all()


@pytest.mark.parametrize("gt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_gradients_at_the_ends_of_the_number_range(ra, d, gt):
    """Rows and gradients whose products leave fp32's range although the results are inside it.

    The tolerance is the one above.  Products of h w and x that fall below 2^-126 are off by at most
    2^-150 each, d of them together by r 2^-150 in the mean: less than 2^-18 of h w = 2^-112 where r <= 2^20
    (eps 1e-6, 1e-22 with its rows scaled), and rows whose sum is below 2^-90 beside a smaller eps are scaled."""
    powers = [(56, 75), (56, 118), (0, 118), (0, -112), (-39, -112), (-39, 100), (-60, -112), (-120, -100), (-130, -100),
              (100, 118), (120, 118), (120, -10), (30, 60), (-20, -112)]
    n, rotary, freq = len(powers), ra.Rotary(d), O.frequencies(d, 10000.0)
    g = torch.Generator().manual_seed(d)
    scale = [torch.tensor([2.0 ** p[i] for p in powers], dtype=torch.float64).view(n, 1, 1) for i in range(2)]
    x = (torch.randn(n, 1, d, generator=g) * scale[0]).to(torch.bfloat16).cuda()
    gy = (torch.randn(n, 1, d, generator=g) * scale[1]).to(gt).cuda()
    pos = torch.arange(n, dtype=torch.int32).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    for eps, fit in ((1e-6, 14), (1e-22, 13), (0.0, 13)):
        want, _ = O.backward(f64(x), f64(gy), pos.cpu().numpy(), freq, False, f64(w), eps)
        rows = (np.abs(want) < 2.0 ** 126).all(axis=(1, 2))      # (the others have no bf16 number, or the last few)
        assert rows.sum() == fit
        dx, _, _, _ = ra.qk_norm_rope_bwd(x, x.clone(), gy, gy.clone(), pos, rotary, w, w, eps=eps)
        check_bwd(dx[rows], None, x[rows], gy[rows], pos[rows], freq, False, w, eps)
        for i in rows.nonzero()[0]:                              # the weights' gradients of each row alone
            one = slice(i, i + 1)
            dx1, _, dw, _ = ra.qk_norm_rope_bwd(x[one], x[one].clone(), gy[one], gy[one].clone(), pos[one], rotary, w, w, eps=eps)
            assert torch.equal(dx1, dx[one])
            check_bwd(dx1, dw, x[one], gy[one], pos[one], freq, False, w, eps)


def test_negative_positions_are_no_tokens(ra):
    q, k, pos, wq, wk = case(60, 4, 2, 128, far=False)
    q[3] = float("nan")
    pos[3] = -1
    pos[5] = -(1 << 31)
    rotary = ra.Rotary(128)
    qo, ko = ra.qk_norm_rope_fwd(q, k, pos, rotary, wq, wk)
    gone = pos < 0
    assert torch.all(qo[gone] == 0) and torch.all(ko[gone] == 0)
    gq, gk = torch.randn_like(qo), torch.randn_like(ko)
    gq[3] = float("nan")
    dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk)
    assert torch.all(dq[gone] == 0) and torch.all(dk[gone] == 0)
    assert torch.isfinite(dwq).all() and torch.isfinite(dwk).all()
    keep = ~gone
    d2 = ra.qk_norm_rope_bwd(q[keep], k[keep], gq[keep], gk[keep], pos[keep], rotary, wq, wk)
    assert torch.equal(dq[keep], d2[0]) and torch.allclose(dwq, d2[2], rtol=1e-4, atol=1e-4)


def test_no_tokens(ra):
    rotary, w = ra.Rotary(64), torch.ones(64).cuda()
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16).cuda() for h in (4, 2))
    pos = torch.empty(0, dtype=torch.int32).cuda()
    qo, ko = ra.qk_norm_rope_fwd(q, k, pos, rotary, w, w)
    assert qo.shape == q.shape and ko.shape == k.shape
    dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(q, k, q, k, pos, rotary, w, w)
    assert torch.all(dwq == 0) and torch.all(dwk == 0)


def test_in_place_and_into_slices(ra):
    """On slices of a fused projection in place, and gradients into slices of its gradient: the rest stays."""
    T, Hq, Hkv, d = 91, 6, 2, 128
    q, k, pos, wq, wk = case(T, Hq, Hkv, d)
    rotary = ra.Rotary(d)
    want = ra.qk_norm_rope_fwd(q, k, pos, rotary, wq, wk)
    qkv = torch.randn(T, Hq + 2 * Hkv, d).to(torch.bfloat16).cuda()
    qkv[:, :Hq], qkv[:, Hq:Hq + Hkv] = q, k
    v = qkv[:, Hq + Hkv:].clone()
    out = ra.qk_norm_rope_fwd(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos, rotary, wq, wk,
                              out=(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]))
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(qkv[:, Hq + Hkv:], v)
    gq, gk = torch.randn_like(want[0]), torch.randn_like(want[1])
    dense = ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk)
    dqkv = torch.full_like(qkv, 7.0)
    ws = ra.qk_norm_rope_workspace(d)
    got = ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk, workspace=ws, out=(dqkv[:, :Hq], dqkv[:, Hq:Hq + Hkv]))
    for a, b in zip(got, dense):
        assert torch.equal(a, b)                                 # the weights' gradients too: one order of addition
    assert torch.all(dqkv[:, Hq + Hkv:] == 7.0)


def test_caller_owned_outputs_allocate_nothing(ra):
    T, Hq, Hkv, d = 91, 6, 2, 128
    q, k, pos, wq, wk = case(T, Hq, Hkv, d)
    rotary, ws = ra.Rotary(d), ra.qk_norm_rope_workspace(d)
    y = ra.qk_norm_rope_fwd(q, k, pos, rotary, wq, wk)
    want = ra.qk_norm_rope_bwd(q, k, *y, pos, rotary, wq, wk)
    fwd, bwd = tuple(map(torch.empty_like, y)), tuple(map(torch.empty_like, want))
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
    before = count()
    ra.qk_norm_rope_fwd(q, k, pos, rotary, wq, wk, out=fwd)
    got = ra.qk_norm_rope_bwd(q, k, *y, pos, rotary, wq, wk, workspace=ws, out=bwd)
    assert count() == before
    assert all(a is b for a, b in zip(got, bwd)) and all(map(torch.equal, got + fwd, want + y))
    some = ra.qk_norm_rope_bwd(q, k, *y, pos, rotary, wq, wk, out=bwd[:2] + (None, bwd[3].zero_()))
    assert some[3] is bwd[3] and all(map(torch.equal, some, want))
    for kw, word in ((dict(out=bwd[:2] + (bwd[2].bfloat16(), None)), "dq_weight has dtype"),
                     (dict(out=bwd[:3] + (torch.empty(2 * d).cuda()[::2],)), "dk_weight must be contiguous"),
                     (dict(out=bwd, weight_grads=False), "not asked for"),
                     (dict(out=bwd[:2] + (torch.empty(64).cuda(), None)), "dq_weight has shape")):
        with pytest.raises(ValueError, match=word):
            ra.qk_norm_rope_bwd(q, k, *y, pos, rotary, wq, wk, workspace=ws, **kw)
    with pytest.raises(ValueError, match="not there"):
        ra.qk_norm_rope_bwd(q, k, *y, pos, rotary, wq, None, workspace=ws, out=bwd)
    with pytest.raises(ra.RingAttnError, match="lies over"):
        ra.qk_norm_rope_bwd(q, k, *y, pos, rotary, wq, wk, workspace=ws, out=bwd[:3] + (bwd[2],))


def test_autograd(ra):
    T, Hq, Hkv, d = 70, 4, 2, 64
    q, k, pos, wq, wk = case(T, Hq, Hkv, d, w=torch.bfloat16, far=False)
    rotary = ra.Rotary(d, 32)
    qkv = torch.cat([q, k, k], dim=1).requires_grad_()
    wq, wk = wq.requires_grad_(), wk.requires_grad_()
    a, b = ra.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos, rotary, wq, wk)
    gq = torch.randn_like(a)
    (a * gq).sum().backward(retain_graph=True)                   # only the queries' result is used
    dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(q, k, gq, torch.zeros_like(b), pos, rotary, wq, wk)
    assert torch.equal(qkv.grad[:, :Hq], dq) and torch.all(qkv.grad[:, Hq:] == 0)
    assert torch.equal(wq.grad, dwq.to(torch.bfloat16)) and torch.all(wk.grad == 0)
    b.sum().backward()                                           # an expanded gradient
    ones = ra.qk_norm_rope_bwd(q, k, torch.zeros_like(a), torch.ones_like(b), pos, rotary, wq, wk)
    assert torch.equal(qkv.grad[:, Hq:Hq + Hkv], ones[1])
    frozen = ra.qk_norm_rope(q, k, pos, rotary, wq.detach(), wk.detach())
    assert not frozen[0].requires_grad


def test_streams_graphs_and_two_calls_at_once(ra):
    T, Hq, Hkv, d = 513, 8, 2, 128
    q, k, pos, wq, wk = case(T, Hq, Hkv, d)
    rotary = ra.Rotary(d)
    gq, gk = torch.randn(T, Hq, d).to(torch.bfloat16).cuda(), torch.randn(T, Hkv, d).to(torch.bfloat16).cuda()
    want, grads = ra.qk_norm_rope_fwd(q, k, pos, rotary, wq, wk), ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(ra.qk_norm_rope_fwd(q, k, pos, rotary, wq, wk) + ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want + grads):
            assert torch.equal(a, b)
    # captured, replayed with other contents of the same buffers
    out, dout, ws = tuple(map(torch.empty_like, want)), tuple(map(torch.empty_like, grads[:2])), ra.qk_norm_rope_workspace(d)
    qs, ks, ps = q.contiguous(), k.contiguous(), pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.qk_norm_rope_fwd(qs, ks, ps, rotary, wq, wk, out=out)
        _, _, dwq, dwk = ra.qk_norm_rope_bwd(qs, ks, gq, gk, ps, rotary, wq, wk, workspace=ws, out=dout)
    for turn in range(2):
        if turn:
            qs.copy_(qs.flip(0))
            ps.copy_(ps.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        f = ra.qk_norm_rope_fwd(qs, ks, ps, rotary, wq, wk)
        b = ra.qk_norm_rope_bwd(qs, ks, gq, gk, ps, rotary, wq, wk)
        for x, y in zip(out + dout + (dwq, dwk), f + b):
            assert torch.equal(x, y)


def test_before_ring_attention(ra):
    """Norm and rotation, ring attention and both backward passes, as a training step runs them.

    Ring attention's gradients differ from the oracle's by roundings of P, dS and the
    results to bf16 (2^-9 of each, of either sign): together less than 2^-6 of their norm, and the
    gradients of rows before the norm are linear in them."""
    d, Hq, Hkv, cu = 64, 4, 2, [0, 96, 256]
    g = torch.Generator().manual_seed(9)
    x = torch.randn(cu[-1], Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16)
    do = torch.randn(cu[-1], Hq, d, generator=g).to(torch.bfloat16)
    w = [(1 + 0.3 * torch.randn(d, generator=g)) for _ in range(2)]
    qkv, wq, wk = x.cuda().requires_grad_(), w[0].cuda().requires_grad_(), w[1].cuda().requires_grad_()
    rotary, freq = ra.Rotary(d, base=500.0), O.frequencies(d, 500.0)
    pos = ra.rope_positions(cu)
    q, k = ra.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos, rotary, wq, wk)
    o, _ = ra.ring_attention(q, k, qkv[:, Hq + Hkv:].contiguous(), cu, 2)
    o.backward(do.cuda())
    scale = 1 / math.sqrt(d)
    rq, rk, rv, ro, _ = A.attention_bwd(q.detach().cpu(), k.detach().cpu(), x[:, Hq + Hkv:], do, cu, True, scale)
    p = pos.cpu().numpy()
    dq, dwq = O.backward(x[:, :Hq].double().numpy(), rq, p, freq, False, w[0].double().numpy(), 1e-6)
    dk, dwk = O.backward(x[:, Hq:Hq + Hkv].double().numpy(), rk, p, freq, False, w[1].double().numpy(), 1e-6)
    for got, want in ((qkv.grad[:, :Hq], dq), (qkv.grad[:, Hq:Hq + Hkv], dk), (qkv.grad[:, Hq + Hkv:], rv), (wq.grad, dwq),
                      (wk.grad, dwk), (o, ro)):
        assert np.linalg.norm(f64(got) - want) <= 2.0 ** -6 * np.linalg.norm(want)


def test_captured_training_step(ra):
    T, Hq, Hkv, d = 130, 4, 2, 128
    q, k, pos, wq, wk = case(T, Hq, Hkv, d, fused=False)
    rotary = ra.Rotary(d)
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    gq, gk = torch.randn_like(q), torch.randn_like(k)

    def step():
        torch.autograd.backward(ra.qk_norm_rope(leaves[0], leaves[1], pos, rotary, leaves[2], leaves[3]), (gq, gk))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t in leaves:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(2):
        with torch.no_grad():
            leaves[0].mul_(1.5)
            gk.neg_()
        graph.replay()
        torch.cuda.synchronize()
        want = ra.qk_norm_rope_bwd(*(t.detach() for t in leaves[:2]), gq, gk, pos, rotary, *(t.detach() for t in leaves[2:]))
        for t, x in zip(leaves, want):
            assert torch.equal(t.grad, x)


def test_offsets_beyond_32_bits(ra):
    """A row far enough behind that its element offset passes 2^31 and its byte offset 2^32."""
    T, Hq, Hkv, d = (1 << 31) // (40 * 128) + 3000, 32, 8, 128
    rotary = ra.Rotary(d)
    q = torch.empty(T, Hq + Hkv, d, dtype=torch.bfloat16, device="cuda").normal_()
    out = torch.empty_like(q)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ra.qk_norm_rope_fwd(q[:, :Hq], q[:, Hq:], pos, rotary, out=(out[:, :Hq], out[:, Hq:]))
    tail = slice(T - 500, T)
    a, b = ra.qk_norm_rope_fwd(q[tail, :Hq], q[tail, Hq:], pos[tail], rotary)
    assert torch.equal(out[tail, :Hq], a) and torch.equal(out[tail, Hq:], b)
    check_fwd(a[:40], q[T - 500:T - 460, :Hq], pos[T - 500:T - 460], O.frequencies(d, 10000.0), False, None, 1e-6)
    out.fill_(3.0)
    g = q.flip(0)
    ra.qk_norm_rope_bwd(q[:, :Hq], q[:, Hq:], g[:, :Hq], g[:, Hq:], pos, rotary, out=(out[:, :Hq], out[:, Hq:]))
    a, b, _, _ = ra.qk_norm_rope_bwd(q[tail, :Hq], q[tail, Hq:], g[tail, :Hq], g[tail, Hq:], pos[tail], rotary)
    assert torch.equal(out[tail, :Hq], a) and torch.equal(out[tail, Hq:], b)


def test_refusals(ra):
    q, k, pos, wq, wk = case(8, 4, 2, 64)
    rotary = ra.Rotary(64)
    call = lambda *a, **kw: ra.qk_norm_rope_fwd(*a, **kw)  # noqa: E731
    for args, word in (((q.float(), k, pos, rotary), "dtype"), ((q, k[:7], pos, rotary), "shapes"),
                       ((q, k, pos.long(), rotary), "positions"), ((q, k, pos[:7], rotary), "positions"),
                       ((q, k, pos, ra.Rotary(128)), "expected"), ((q, k, pos, ra.Rotary(64, device="cpu")), "rotary"),
                       ((q, k, pos, rotary, wq[:32]), "q_weight"), ((q, k, pos, rotary, wq.half()), "dtype"),
                       ((q, k, pos, rotary, wq, wk.bfloat16()), "k_weight"),
                       ((q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, rotary), "one after the other")):
        with pytest.raises(ValueError, match=word):
            call(*args)
    with pytest.raises(ValueError, match="norm"):
        call(q, k, pos, rotary, wq, wk, eps=None)
    with pytest.raises(ra.RingAttnError, match="lies over"):
        call(q, k, pos, rotary, out=(q, q[:, :2]))
    with pytest.raises(ra.RingAttnError, match="stride"):
        call(q[:1].expand(8, 4, 64), k, pos, rotary)
    gq, gk = torch.randn(8, 4, 64).cuda(), torch.randn(8, 2, 64).cuda()
    with pytest.raises(ValueError, match="gk has dtype"):
        ra.qk_norm_rope_bwd(q, k, gq, gk.bfloat16(), pos, rotary)
    with pytest.raises(ValueError, match="gq has dtype"):
        ra.qk_norm_rope_bwd(q, k, gq.half(), gk.half(), pos, rotary)
    with pytest.raises(ra.RingAttnError, match="workspace"):
        ra.qk_norm_rope_bwd(q, k, gq, gk, pos, rotary, wq, wk, workspace=torch.empty(256, dtype=torch.uint8).cuda())
