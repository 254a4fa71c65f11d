"""Plain 64-bit implementations of the serving operators (test infrastructure, numpy only).

Written from the definitions, one token, head or row at a time, sharing no code with the library.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
#: unit roundoff of the 16-bit types (11 and 8 significant bits)
ROUNDOFF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
#: half the spacing of their subnormals
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def e4m3_values():
    """The 256 codes' values: sign, 4 exponent bits (bias 7), 3 fraction bits; all ones is NaN."""
    out = np.empty(256)
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 127) == 127 else (-x if s else x)
    return out


def e4m3_codes(x):
    """Codes of the nearest e4m3 values of x (|x| <= 448; ties to the code with an even fraction); NaN where x is."""
    x = np.asarray(x, dtype=np.float64)
    grid = e4m3_values()[:127]                      # 0 .. 448, ascending
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(np.isfinite(x), code, np.where(np.signbit(x), 255, 127)).astype(np.uint8)


def cache_scale(x):
    """The power of two of one head vector x: least e >= -126 with max |x| <= 448 * 2^e over the finite values."""
    a = np.abs(x[np.isfinite(x)])
    most = a.max() if a.size else 0.0
    if most == 0:
        return 1.0
    e = -126
    while most > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def attention(q, k, v, scale, causal=True, window=0):
    """One sequence, one query head group: q [n][heads][dim], k, v [len][kv][dim] (64 bits) ->
    (o [n][heads][dim], sum_j p_j |v_j| [n][heads][dim], largest sum of |scale q k| over a row's scores [n][heads])."""
    n, heads, _ = q.shape
    length, kv, dv = v.shape
    o, a = np.zeros((n, heads, dv)), np.zeros((n, heads, dv))
    big = np.zeros((n, heads))
    for i in range(n):
        p = length - n + i
        seen = [j for j in range(length) if (not causal or j <= p) and (window == 0 or j > p - window)]
        if not seen:
            continue
        for h in range(heads):
            g = h // (heads // kv)
            s = scale * (k[seen, g] @ q[i, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            o[i, h] = w @ v[seen, g]
            a[i, h] = w @ np.abs(v[seen, g])
            big[i, h] = (np.abs(scale * k[seen, g]) @ np.abs(q[i, h])).max()
    return o, a, big


def quant_weights(codes, scales, zeros, K, group):
    """(codes - zeros [M][K] whole numbers, scales [M][K]) of a packed matrix, column by column."""
    M = codes.shape[0]
    c, s = np.empty((M, K)), np.empty((M, K))
    for k in range(K):
        z = 8 if zeros is None else zeros[:, k // group].astype(np.int64) & 15
        c[:, k] = ((codes[:, k // 2].astype(np.int64) >> (4 * (k % 2))) & 15) - z
        s[:, k] = scales[:, k // group]
    return c, s
