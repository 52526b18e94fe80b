"""Oracle for the serving operators: rotary positions, the paged K/V cache
(quantised by rows) and attention of drafted tokens over it.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Plain float64, one
sequence and head at a time; float32 only where the definition decides codes
or scales in float32.
"""

import math

import numpy as np

from .fp8 import E4M3_MAX, e4m3_decode, e4m3_encode

__all__ = ["rope_ref", "quantize_rows", "dequantize_rows", "gather_rows", "ref_tree"]

_AMAX_MIN = np.float32(E4M3_MAX * 2.0 ** -126)


def rope_ref(x, positions, inv_freq, interleaved=False, factor=1.0, sign=1.0):
    """x [..., N, d] rotated by positions [N] (float64; sign -1: the gradient)."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        theta = np.asarray(positions, dtype=np.float64) * float(inv_freq[i]) * sign
        c, s = np.cos(theta), np.sin(theta)
        y[..., a] = factor * (x[..., a] * c - x[..., b] * s)
        y[..., b] = factor * (x[..., b] * c + x[..., a] * s)
    return y


def quantize_rows(x):
    """Rows of x [..., d] (fp32-exact) as (e4m3 codes uint8, scale float32).

    top = max(amax, 448 * 2^-126); scale = top / 448 (1 for a row of zeros) and
    448 / top, x * (448 / top) in fp32; a row that is not finite has scale NaN
    (its codes are unspecified, 0 here).
    """
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad[..., None], np.float32(0), x)
    top = np.maximum(np.where(bad, np.float32(0), amax), _AMAX_MIN).astype(np.float32)
    inv = np.float32(E4M3_MAX) / top
    codes = e4m3_encode((safe * inv[..., None]).astype(np.float32).astype(np.float64))
    scale = np.where(amax > 0, top / np.float32(E4M3_MAX), np.float32(1)).astype(np.float32)
    scale = np.where(bad, np.float32(np.nan), scale).astype(np.float32)
    return codes, scale


def dequantize_rows(codes, scale):
    """float64 values of rows of codes [..., d] with scales [...]."""
    return e4m3_decode(codes) * np.asarray(scale, dtype=np.float64)[..., None]


def gather_rows(pool, table, head, start, count):
    """Positions start .. start + count - 1 of one sequence and head: pool
    [pages, Hk, page_size, ...], table the sequence's pages."""
    page = pool.shape[2]
    return np.stack([pool[table[j // page], head, j % page] for j in range(start, start + count)]) \
        if count else np.zeros((0,) + pool.shape[3:], dtype=pool.dtype)


def ref_tree(q, k, v, ctx, mask, scale):
    """O [T, d], LSE [T] and sum_j p_j |v_j| [T, d] of queries q [T, d] over
    keys k, v [ctx + n, d] (float64): query t sees j < ctx, and j = ctx + u if
    mask[t, u].  Keys that are not seen are left out altogether."""
    q = np.asarray(q, dtype=np.float64)
    T, n = q.shape[0], len(k) - ctx
    o, spread = np.zeros((T, v.shape[1])), np.zeros((T, v.shape[1]))
    lse = np.full(T, -np.inf)
    for t in range(T):
        seen = np.concatenate([np.ones(ctx, bool), np.asarray(mask)[t, :n] != 0])
        if not seen.any():
            continue
        s = scale * (k[seen] @ q[t])
        m = s.max()
        if m == -np.inf:
            continue
        p = np.exp(s - m)
        lse[t] = m + math.log(p.sum())
        p = p / p.sum()
        o[t] = p @ v[seen]
        spread[t] = p @ np.abs(v[seen])
    return o, lse, spread
