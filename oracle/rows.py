"""RMS norm of query and key heads and their rotation by position, float64 CPU
oracle: the forward and its gradients.

The operations are this library's own (the source pages take q and k as they
are); ``include/bsa.h`` states them.

TEST INFRASTRUCTURE: see the package docstring for who may import this.
"""

from __future__ import annotations

import numpy as np


def _pairs(r, interleaved):
    j = np.arange(r // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + r // 2)


def turn(x, pos, inv_freq, interleaved, scale=1.0, back=False):
    """Rows x [B, H, T, D] at positions pos [B, T], turned (or turned back) and scaled; elements past the pairs stay."""
    x = np.array(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    a, b = _pairs(2 * len(f), interleaved)
    ang = np.asarray(pos, dtype=np.float64)[:, None, :, None] * f * (-1.0 if back else 1.0)
    c, s = np.cos(ang) * scale, np.sin(ang) * scale
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = xa * c - xb * s, xa * s + xb * c
    return x


def reach(x, inv_freq, interleaved, scale=1.0):
    """What an element's rounding errors go by: |x_a| + |x_b| of its pair, times the scale (|x| past the pairs)."""
    x = np.abs(np.array(x, dtype=np.float64))
    a, b = _pairs(2 * len(inv_freq), interleaved)
    both = (x[..., a] + x[..., b]) * abs(scale)
    x[..., a] = x[..., b] = both
    return x


def norm(x, w, eps):
    """(r x, r) of rows x [..., D]; (x, 1) without weights."""
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x, np.ones((*x.shape[:-1], 1))
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def forward(x, w, pos, inv_freq, interleaved, scale, eps):
    """``(y, e)``: the result, and ``reach`` of the normalised rows."""
    h, _ = norm(x, w, eps)
    n = h if w is None else h * np.asarray(w, dtype=np.float64)
    return turn(n, pos, inv_freq, interleaved, scale), reach(n, inv_freq, interleaved, scale)


def backward(x, dy, w, pos, inv_freq, interleaved, scale, eps):
    """``(dx, dw, ex, ew)``; ex and ew bound what the errors of dx and dw go by (dw and ew None without weights)."""
    dy = np.asarray(dy, dtype=np.float64)
    g, eg = turn(dy, pos, inv_freq, interleaved, scale, back=True), reach(dy, inv_freq, interleaved, scale)
    if w is None:
        return g, None, eg, None
    w = np.asarray(w, dtype=np.float64)
    h, r = norm(x, w, eps)
    dx = r * (g * w - h * (g * w * h).mean(-1, keepdims=True))
    ex = r * (eg * np.abs(w) + np.abs(h) * (eg * np.abs(w * h)).mean(-1, keepdims=True))
    return dx, (g * h).sum((0, 1, 2)), ex, (eg * np.abs(h)).sum((0, 1, 2))
