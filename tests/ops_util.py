"""float64 forms of the cache operators (include/csa2_ops.h), in numpy: norm
and rotation, dense attention, attention weight, eviction."""
from __future__ import annotations

import numpy as np


def freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / max(rot, 1))


def norm_rope(x, w, eps, pos, fr, interleaved):
    """x [n, ..., D] float64 -> (y, spread): spread is |u| + |v| of each
    channel's pair (|y| where nothing is rotated), the size that rounding
    errors of the rotation scale with."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    h, D = len(fr), x.shape[-1]
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(fr, np.float64)
    a = a.reshape(a.shape[0], *([1] * (x.ndim - 2)), h)
    i = np.arange(h)
    lo = D - 2 * h
    p, q = (lo + 2 * i, lo + 2 * i + 1) if interleaved else (lo + i, lo + h + i)
    out, spread = y.copy(), np.abs(y)
    u, v = y[..., p], y[..., q]
    out[..., p], out[..., q] = u * np.cos(a) - v * np.sin(a), u * np.sin(a) + v * np.cos(a)
    spread[..., p] = spread[..., q] = np.abs(u) + np.abs(v)
    return out, spread
