"""fp64 restatement of the 4-bit key/value cache.  TEST INFRASTRUCTURE ONLY.

Shares no code with the library: the two number formats are tables of their
values, rounding is "nearest entry, ties to the even code", the page
bookkeeping is Python lists, and attention is written out row by row.
"""

import numpy as np

GROUP = 16
ELEMENTS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# scale codes 0..226: no sign, 5 exponent bits (bias 15), 3 mantissa bits, up to 10240
SCALES = np.array([m * 2.0 ** -17 for m in range(8)]
                  + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 29) for m in range(8)])
SCALES = SCALES[SCALES <= 10240]


def nearest(x, table):
    """Index of the entry of `table` nearest to x >= 0; a tie goes to the even index."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def rounded(x):
    """Values that the cache holds for rows x [..., d] (float64 in and out)."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    amax = np.abs(g).max(-1, keepdims=True)
    ok = np.isfinite(amax)
    s = SCALES[nearest(np.where(ok, amax, 0) / 6.0, SCALES)]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, np.abs(g) / s, 0.0)
        v = np.sign(g) * ELEMENTS[nearest(np.where(ok, y, 0), ELEMENTS)] * s
    return np.where(ok, v, np.nan).reshape(x.shape)


def tables(kv_lens, new_lens, table, page, num_slots, free=None, count=0):
    """(lens, cu, slots, positions, count, table, free) after a step, or None if it cannot be done."""
    table = [list(r) for r in table]
    free = None if free is None else list(free)
    width = len(table[0])
    pages = lambda n: -(-n // page)
    for n, a in zip(kv_lens, new_lens):
        if n < 0 or a < -1 or n + max(a, 0) > width * page:
            return None
    if free is not None:
        back = [table[r][j] for r, a in enumerate(new_lens) if a < 0 for j in range(pages(kv_lens[r]))]
        if count < 0 or count + len(back) > len(free):
            return None
        free[count:count + len(back)] = back
        count += len(back)
        if sum(pages(n + a) - pages(n) for n, a in zip(kv_lens, new_lens) if a > 0) > count:
            return None
    lens, cu, slots, pos = [], [0], [], []
    for r, (n, a) in enumerate(zip(kv_lens, new_lens)):
        if a >= 0 and free is not None:
            for j in range(pages(n), pages(n + a)):
                count -= 1
                table[r][j] = free[count]
        for t in range(n, n + max(a, 0)):
            pg = table[r][t // page]
            slots.append(-1 if pg < 0 else pg * page + t % page)
            pos.append(t)
        lens.append(0 if a < 0 else n + a)
        cu.append(cu[-1] + max(a, 0))
    if len(slots) > num_slots:
        return None
    pad = [-1] * (num_slots - len(slots))
    return lens, cu, slots + pad, pos + pad, count, table, free


def attention(q, keys, values, kv_lens, cu_q, causal, scale):
    """o [T, Hq, d] and lse [Hq, T] in float64; keys[r], values[r] are [L_r, Hkv, d]."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, d = q.shape
    o, lse = np.zeros((T, Hq, d)), np.full((Hq, T), -np.inf)
    for r, L in enumerate(kv_lens):
        n = cu_q[r + 1] - cu_q[r]
        G = Hq // keys[r].shape[1]
        for h in range(Hq):
            k, v = keys[r][:L, h // G], values[r][:L, h // G]
            for i in range(n):
                see = min(L, max(0, L - n + i + 1)) if causal else L
                if see == 0:
                    continue
                t = cu_q[r] + i
                s = scale * (k[:see] @ q[t, h])
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                o[t, h] = (p / z) @ v[:see]
                lse[h, t] = m + np.log(z)
    return o, lse
