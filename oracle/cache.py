"""Oracle of the 4-bit cache and of eviction by accumulated attention weight: numpy in float64,
written from the definitions in include/rkv.h, without the library's arithmetic.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # e2m1
MAX_SCALE_BYTE = 226
MAX_VALUE = 61440.0


def scale_number(byte):
    """The number of a scale byte: 5 exponent and 3 mantissa bits, bias 15, subnormals at 0."""
    byte = np.asarray(byte, dtype=np.int64)
    e, m = byte >> 3, byte & 7
    return np.where(e == 0, m * 2.0 ** -17, (1 + m / 8.0) * 2.0 ** (e - 15.0))


def _nearest(x, grid):
    """Index of the nearest number of an ascending grid; a tie goes to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def kv4_quantise(x):
    """[.., 128] numbers -> codes [.., 64] and scale bytes [.., 8]."""
    x = np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf)
    x = np.clip(x, -MAX_VALUE, MAX_VALUE)
    blocks = x.reshape(x.shape[:-1] + (8, 16))
    sb = _nearest(np.abs(blocks).max(-1) / 6.0, scale_number(np.arange(MAX_SCALE_BYTE + 1)))
    s = scale_number(sb)[..., None]
    safe = np.where(s > 0, s, 1.0)
    code = np.where(s > 0, _nearest(np.minimum(np.abs(blocks) / safe, 6.0), MAGNITUDES), 0)
    code = (code + 8 * np.signbit(blocks)).reshape(x.shape)
    return (code[..., 0::2] + 16 * code[..., 1::2]).astype(np.uint8), sb.astype(np.uint8)


def kv4_values(codes, scales):
    """[.., 64] codes and [.., 8] scale bytes -> the numbers [.., 128] they stand for."""
    codes = np.asarray(codes, dtype=np.int64)
    pair = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (128,))
    v = np.where(pair & 8, -1.0, 1.0) * MAGNITUDES[pair & 7]
    return v * np.repeat(scale_number(scales), 16, axis=-1)


def softmax_weights(q, k, scale, visible=None):
    """Softmax rows [R, T] of q [R, d] over k [T, d]; visible [R, T] masks keys. A row that sees
    nothing is zero."""
    s = (np.asarray(q, dtype=np.float64) @ np.asarray(k, dtype=np.float64).T) * scale
    if visible is not None:
        s = np.where(visible, s, -np.inf)
    if s.shape[1] == 0:
        return s
    m = s.max(1, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    total = e.sum(1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def decode_weights(q, k, v, scale):
    """One decode step of a KV group: outputs [G, d] and the weight of each token [T]."""
    p = softmax_weights(q, k, scale)
    return p @ np.asarray(v, dtype=np.float64), p.sum(0)


def prompt_weights(q, k, scale):
    """q [G, T, d], k [L, d], the queries at the last T positions -> weights [L]."""
    G, T, d = q.shape
    L = k.shape[0]
    pos = np.arange(L - T, L)
    seen = np.tile(np.arange(L)[None, :] <= pos[:, None], (G, 1))
    return softmax_weights(q.reshape(G * T, d), k, scale, seen).sum(0)


def evict(weights, pos, seen, keep, recent):
    """weights, pos of one (unit, KV head)'s L rows -> (source row of every kept row, its
    position); rows and positions unchanged when L <= keep."""
    L = len(weights)
    rows = np.arange(L)
    if L <= keep:
        return rows, np.asarray(pos).copy()
    at = np.where(np.asarray(pos) >= 0, pos, seen - (L - rows))
    key = np.where(at >= seen - recent, np.inf, np.nan_to_num(weights, nan=np.finfo(float).max))
    kept = np.zeros(L, dtype=bool)
    kept[np.lexsort((rows, -key))[:keep]] = True
    src = rows[:keep].copy()
    src[~kept[:keep]] = rows[keep:][kept[keep:]]
    return src, at[src]
