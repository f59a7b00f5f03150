"""Plain fp64 paged cache and its attention on the CPU (numpy).

A sequence's positions are looked up one page at a time through its table and
everything is computed from the definitions; the split of the heads over ranks
only decides which arrays are passed.
"""
from __future__ import annotations

import numpy as np


def e4m3_values():
    """The 256 codes' values (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 0x7F == 0x7F else (-x if c & 0x80 else x)
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # codes 0 .. 126 in rising order


def quantise(x):
    """Rows [..., d] as (codes uint8, power bytes uint8): see fcc_cache in fcc.h."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0).max(axis=-1)
    k = np.full(a.shape, -64)
    while (big := a > 448 * 2.0 ** k).any():
        k = np.where(big, k + 1, k)
    y = np.abs(x) * (2.0 ** -k)[..., None]
    mid = (_POSITIVE[:-1] + _POSITIVE[1:]) / 2  # halfway to the next code
    lo = np.searchsorted(mid, np.where(np.isfinite(y), y, 0), side="left")  # codes with mid < y
    tie = np.isin(y, mid) & (lo % 2 == 1)  # a tie goes to the even code
    codes = np.where(np.isfinite(y), lo + tie, 0x7F).astype(np.uint8)
    neg = np.signbit(x) & np.isfinite(x)
    return codes | np.where(neg, 0x80, 0).astype(np.uint8), (k + 127).astype(np.uint8)


def values(codes, power):
    return _VALUES[codes] * (2.0 ** (power.astype(np.float64) - 127))[..., None]


def rows_of(pool, table_row, first, last):
    """Positions first .. last - 1 of a pool [pages, H, P, d]: [last - first, H, d]."""
    P = pool.shape[2]
    return np.array([pool[table_row[j // P], :, j % P] for j in range(first, last)]).reshape(
        last - first, pool.shape[1], -1)


def attention(Q, keys, vals, length, scale, window=0):
    """Rows Q [n, Hq, d] at the last n of `length` positions; keys, vals [length, H, d] (those that
    no row sees are not touched).  Returns O [n, Hq, d], lse [n, Hq] and sum softmax |v| [n, Hq, d]."""
    n, Hq, d = Q.shape
    O, A = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse = np.full((n, Hq), -np.inf)
    if length < n:
        return O, lse, A
    G = Hq // keys.shape[1]
    for i in range(n):
        p = length - n + i
        lo = max(0, p - window + 1) if window else 0
        for h in range(Hq):
            k, v = keys[lo:p + 1, h // G], vals[lo:p + 1, h // G]
            s = scale * (k @ Q[i, h])
            m = s.max()
            e = np.exp(s - m)
            O[i, h], A[i, h] = e @ v / e.sum(), e @ np.abs(v) / e.sum()
            lse[i, h] = m + np.log(e.sum())
    return O, lse, A
