"""Float64 definitions of rotary positions and of the paged cache: append, decode (TEST INFRASTRUCTURE).

Plain loops over tokens, rows and heads, sharing no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from . import attend

# e4m3 by its bits: 1 sign, 4 exponent (bias 7), 3 mantissa; 0x7F is NaN, there are no infinities, 448 is the largest
_MAG = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) if (e, m) != (15, 7) else np.nan
                 for e in range(16) for m in range(8)])


def e4m3_to_f64(bits) -> np.ndarray:
    b = np.asarray(bits).astype(np.uint8)
    return np.where(b & 0x80, -_MAG[b & 0x7F], _MAG[b & 0x7F])


def f64_to_e4m3(x) -> np.ndarray:
    """Bits of the nearest e4m3 value (ties to the even mantissa), at most 448 in size; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    ax = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), 448.0)
    up = np.clip(np.searchsorted(_MAG[:127], ax), 0, 126)          # the first value that is not below
    down = np.maximum(up - 1, 0)
    lo, hi = ax - _MAG[down], _MAG[up] - ax
    near = np.where((hi < lo) | ((hi == lo) & (up % 2 == 0)), up, down)
    out = np.where(np.isnan(x), 0x7F, near).astype(np.uint8)
    return out | (np.signbit(x).astype(np.uint8) << 7)


def rotate(x, pos, inv_freq, layout: str, factor: float = 1.0, inverse: bool = False):
    """(values, sizes) of x [n, heads, d] float64 turned by pos * inv_freq: sizes is |x_a| + |x_b| of a value's pair,
    times |factor| (0 where nothing turns), which the tolerances scale with."""
    y, size = np.array(x, dtype=np.float64), np.zeros(np.shape(x))
    half = len(inv_freq)
    for j in range(half):
        a, b = (j, j + half) if layout == "half" else (2 * j, 2 * j + 1)
        t = np.asarray(pos, dtype=np.float64) * float(inv_freq[j])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None] * (-1.0 if inverse else 1.0)
        y[:, :, a] = factor * (x[:, :, a] * c - x[:, :, b] * s)
        y[:, :, b] = factor * (x[:, :, b] * c + x[:, :, a] * s)
        size[:, :, a] = size[:, :, b] = abs(factor) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    return y, size


def append(x, pos, row, hq: int, hkv: int, table, page: int, inv_freq=None, layout="half", factor=1.0,
           k_scale=None, v_scale=None):
    """x [n, hq + 2 hkv, d] float64.  Returns (q, size of q's pairs, places): a place is (page, slot, key value
    [hkv, d], its size, value [hkv, d]) of a token that has one, before the rounding to the pages' type."""
    qk, size = (x[:, :hq + hkv], np.zeros_like(x[:, :hq + hkv])) if inv_freq is None \
        else rotate(x[:, :hq + hkv], pos, inv_freq, layout, factor)
    ks = np.ones(hkv) if k_scale is None else np.asarray(k_scale, dtype=np.float64)
    vs = np.ones(hkv) if v_scale is None else np.asarray(v_scale, dtype=np.float64)
    places = []
    for t, p in enumerate(pos):
        if not 0 <= p < page * table.shape[1]:
            continue
        r = t if row is None else int(row[t])
        if 0 <= r < len(table) and table[r][p // page] >= 0:
            places.append((int(table[r][p // page]), int(p) % page, qk[t, hq:] / ks[:, None], size[t, hq:] / ks[:, None],
                           x[t, hq + hkv:] / vs[:, None]))
    return qk[:, :hq], size[:, :hq], places


def decode(q, k, v, table, pos, win: int, scale: float, k_scale=None, v_scale=None) -> np.ndarray:
    """q [rows, hq, d], k / v [pages, page, hkv, d] float64 as stored, table [rows, most].  A page outside the pool
    reads as zeros; a row without keys gives zeros."""
    rows, hq, d = q.shape
    pages, page, hkv, _ = k.shape
    G = hq // hkv
    out = np.zeros((rows, hq, d))
    for r in range(rows):
        p = min(int(pos[r]), page * table.shape[1] - 1)
        if p < 0:
            continue
        at = np.arange(max(0, p - win + 1) if win > 0 else 0, p + 1)
        ids, slot = np.asarray(table[r])[at // page], at % page
        there = (ids >= 0) & (ids < pages)
        for g in range(hkv):
            kk, vv = (np.where(there[:, None], x[np.where(there, ids, 0), slot, g], 0.0) for x in (k, v))
            ks = 1.0 if k_scale is None else float(k_scale[g])
            vs = 1.0 if v_scale is None else float(v_scale[g])
            hs = slice(g * G, g * G + G)
            out[r, hs] = attend(q[r, hs], kk, vv, scale * ks)[0] * vs
    return out
