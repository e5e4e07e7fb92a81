"""Norms of query and key rows with the position rotation, in float64, row by row.

Written from the formulas; shares no code with the GPU path.
"""

import numpy as np


def frequencies(rotary_dim, base):
    return np.array([float(base) ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)])


def pairs(rotary_dim, interleaved):
    """Index arrays (a, b) of the elements that turn together."""
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def rotated(u, positions, freq, interleaved, back=False):
    """Rows u [T, H, d], turned by their positions (``back``: by the opposite angle)."""
    a, b = pairs(2 * len(freq), interleaved)
    angle = np.asarray(positions, dtype=np.float64)[:, None, None] * freq * (-1.0 if back else 1.0)
    c, s = np.cos(angle), np.sin(angle)
    y = u.copy()
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., b] * c + u[..., a] * s
    return y


def forward(x, positions, freq, interleaved, w=None, eps=None):
    """x [T, H, d] float64; eps None: no norm.  Rows at a negative position are zero."""
    u = x
    if eps is not None:
        with np.errstate(all="ignore"):
            u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        u = u if w is None else u * w
    y = rotated(u, positions, freq, interleaved)
    y[np.asarray(positions) < 0] = 0.0
    return y


def backward(x, g, positions, freq, interleaved, w=None, eps=None):
    """(dx, dw) of sum(g y)."""
    g = np.where((np.asarray(positions) < 0)[:, None, None], 0.0, g)
    h = rotated(g, positions, freq, interleaved, back=True)
    if eps is None:
        return h, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    live = (np.asarray(positions) >= 0)[:, None, None]
    dw = (h * np.where(live, n, 0.0)).sum((0, 1))
    hw = h if w is None else h * w
    dx = r * (hw - n * (hw * n).mean(-1, keepdims=True))
    return np.where(live, dx, 0.0), dw
