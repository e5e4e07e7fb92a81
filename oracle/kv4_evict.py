"""Attention weights of cached tokens, and eviction by them, in plain loops and float64.

Written from the definitions; shares no code with the GPU path.
"""

import numpy as np


def weights(q, keys, kv_lens, cu_q, lse, causal, scale):
    """Per request: float64 [L] sums of exp(scale q . k - lse) over the rows and heads that see the key.

    q [T, Hq, d], keys[r] [L_r, Hkv, d], lse [Hq, T].  Rows with lse = -inf see no key.
    """
    out = []
    Hq = q.shape[1]
    for r, L in enumerate(kv_lens):
        n, b = cu_q[r + 1] - cu_q[r], cu_q[r]
        w = np.zeros(L)
        if n and L:
            G = Hq // keys[r].shape[1]
            last = L - n + np.arange(n) if causal else np.full(n, L - 1)
            see = np.arange(L) <= last[:, None]
            for h in range(Hq):
                row = lse[h, b:b + n, None]
                with np.errstate(all="ignore"):
                    p = np.exp(scale * (q[b:b + n, h] @ keys[r][:, h // G].T) - row)
                p = np.where(see & ~np.isneginf(row), p, 0.0)
                w = w + p.sum(0)
        out.append(w)
    return out


def evict(weights, table, kv_lens, budgets, page, max_moves, slack, recent, sinks, free=None, count=0):
    """(lens, dropped, src, dst, count, free, refused) after one call; ``refused``: requests left alone.

    weights: per slot.  A request longer than budget + slack keeps its first
    ``sinks``, last ``recent`` and otherwise heaviest tokens (the lower index first
    among equals; what is no positive number counts as 0).
    """
    slots = len(weights)
    free = None if free is None else list(free)
    lens, dropped, src, dst, refused = [], [], [], [], []
    back = []
    for r, L in enumerate(kv_lens):
        B = budgets[r]
        s, d = [-1] * max_moves, [-1] * max_moves
        new = L
        pages = -(-L // page) if L > 0 else 0
        if L < 0 or L > len(table[r]) * page:
            refused.append(r)
        elif B >= 0 and L > B + slack:
            if B < sinks + recent or any(not 0 <= table[r][j] < slots // page for j in range(pages)):
                refused.append(r)
            else:
                slot = [table[r][i // page] * page + i % page for i in range(L)]
                value = [w if w > 0 else 0.0 for w in (float(weights[x]) for x in slot)]
                middle = sorted(range(sinks, L - recent), key=lambda i: (-value[i], i))[:B - sinks - recent]
                kept = set(range(sinks)) | set(range(L - recent, L)) | set(middle)
                holes = [i for i in range(B) if i not in kept]
                movers = sorted(i for i in kept if i >= B)
                assert len(holes) == len(movers)
                if len(holes) > max_moves:
                    refused.append(r)
                else:
                    for m, (h, i) in enumerate(zip(holes, movers)):
                        s[m], d[m] = slot[i], slot[h]
                    new = B
                    back += [table[r][j] for j in range(-(-B // page), pages)]
        lens.append(new)
        dropped.append(L - new)
        src.append(s)
        dst.append(d)
    if free is not None:
        free[count:count + len(back)] = back
        count += len(back)
    return lens, dropped, src, dst, count, free, refused
