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


# ------------------------------------------------------- dense attention ----

def random_cache(csa2, lens, page, seed, spare_pages=2, scale_codes=(40, 72)):
    """A cache of random packed rows in shuffled pages.  Scales are drawn from
    E4M3 codes of moderate size; rows that no request sees hold arbitrary
    bytes (NaN scale codes among them), and unused table slots -1."""
    import torch
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for n in lens]
    num = sum(per) + spare_pages
    ids = rng.permutation(num).astype(np.int32)
    width = max(1, max(per))
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, p in enumerate(per):
        table[b, :p] = ids[at:at + p]
        at += p
    cache = csa2.Cache(num, page, table, lens)
    codes = rng.integers(0, 256, (num * page, 256), dtype=np.uint8)
    scales = rng.integers(0, 256, (num * page, 32), dtype=np.uint8)
    for b, n in enumerate(lens):
        rows = rows_of(table, page, b, n)
        scales[rows] = rng.integers(*scale_codes, (n, 32), dtype=np.uint8)
    cache.kv_codes.copy_(torch.from_numpy(codes))
    cache.kv_scales.copy_(torch.from_numpy(scales))
    return cache, table, codes, scales


def rows_of(table, page, b, n):
    t = np.arange(n)
    return table[b, t // page].astype(np.int64) * page + t % page


def keys(table, page, codes, scales, b, n):
    """Rows 0 .. n-1 of request b in float64."""
    from oracle import formats as F
    r = rows_of(table, page, b, n)
    return F.dequantize_main_kv(codes[r], scales[r])


def attention(q, K, seen, scale):
    """q [n, H, 512], K [e, 512], seen [n] -> dict of the output, lse, the
    probabilities, sum_e p |v| and sum_c |q_c k_c| (its largest over the
    entries), all float64."""
    s = np.einsum("ihc,ec->ihe", q, K) * scale
    mask = np.arange(K.shape[0])[None, None, :] < np.asarray(seen)[:, None, None]
    s = np.where(mask, s, -np.inf)
    m = s.max(-1, initial=-np.inf)
    p = np.where(mask, np.exp(s - np.where(np.isfinite(m), m, 0.0)[..., None]), 0.0)
    l = p.sum(-1)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, m + np.log(l), -np.inf)
    p = p / np.where(l > 0, l, 1.0)[..., None]
    size = np.abs(scale) * np.einsum("ihc,ec->ihe", np.abs(q), np.abs(K))
    return {"out": np.einsum("ihe,ec->ihc", p, K), "lse": lse, "p": p, "s": s,
            "abs": np.einsum("ihe,ec->ihc", p, np.abs(K)), "size": size.max(-1, initial=0.0)}


def attention_bounds(ref, n_keys):
    """Bounds of the kernels' errors, from their arithmetic alone.
    Scores: 512 products, exact in fp32 (11 by 6 bits), summed in fp32 with
    each partial sum off by at most 2^-23 of the sum of magnitudes; the scaling
    and the subtraction of the maximum add 2 roundings of values no larger:
      d = (512 + 4) 2^-23 sum|q k|.
    A probability and the sum it is divided by are each off by e^d - 1 <= 2 d
    (d < 1), by exp2 (2 units of 2^-23) and the rescaling products (1 unit for
    each of the n/64 steps); P is rounded to fp16 (2^-11, and 2^-24 of the
    row's maximum where it falls below fp16's normal range: at most n 2^-24 of
    sum p|v| spread over n keys); P V adds n partial sums off by 2^-23 each.
    """
    d = (512 + 4) * 2.0 ** -23 * ref["size"]
    assert (d < 1).all()
    rel = 4 * d + 2.0 ** -11 + (2 * n_keys + n_keys / 32 + 8) * 2.0 ** -23
    out = rel[..., None] * ref["abs"] + 2.0 ** -24 * n_keys * ref["abs"].max(-1, keepdims=True, initial=0.0)
    lse = d + (2 * n_keys + 16) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0))
    return out, lse
