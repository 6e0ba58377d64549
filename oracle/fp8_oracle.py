"""fp64 CPU oracle of the 8-bit operators (E4M3 codes, scales per 128).

TEST INFRASTRUCTURE ONLY, like moe_oracle: numpy, no code shared with the CUDA
library.  E4M3 (OCP 8-bit floating point, E4M3 without infinities): sign,
4 exponent bits (bias 7), 3 mantissa bits; 0x7f / 0xff are NaN, the largest
magnitude is 448.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
MAX = 448.0
MIN_SCALE = 2.0 ** -126


def _table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if c & 0x7f == 0x7f:
            v = np.nan
        t[c] = -v if c & 0x80 else v
    return t


E4M3 = _table()


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def decode(codes):
    return E4M3[np.asarray(codes, np.uint8)]


def encode(v):
    """Nearest E4M3 code of each value, ties to the even code, saturating."""
    v = np.asarray(v, np.float64)
    mags = E4M3[:127]                                   # codes 0 .. 126 ascending
    a = np.minimum(np.abs(v), MAX)
    hi = np.searchsorted(mags, np.where(np.isnan(a), 0, a), side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(v), 0x7F, pick) | np.where(np.signbit(v), 0x80, 0)
    return code.astype(np.uint8)


def dequant_rows(q, s):
    """codes [rows, K], scales [rows, blocks(K)] -> float64 [rows, K]."""
    q = np.asarray(q)
    return decode(q) * np.repeat(np.asarray(s, np.float64), BLOCK, axis=-1)[..., :q.shape[-1]]


def dequant_mats(q, s):
    """codes [.., N, K], scales [.., blocks(N), blocks(K)] -> float64."""
    q = np.asarray(q)
    s = np.repeat(np.asarray(s, np.float64), BLOCK, axis=-1)[..., :q.shape[-1]]
    return decode(q) * np.repeat(s, BLOCK, axis=-2)[..., :q.shape[-2], :]


def scales(v):
    """float64 rows [rows, n] -> scales [rows, blocks(n)] (NaN left out)."""
    n = v.shape[1]
    p = np.zeros((v.shape[0], blocks(n) * BLOCK))
    p[:, :n] = np.where(np.isnan(v), 0.0, np.abs(v))
    return np.maximum(p.reshape(v.shape[0], -1, BLOCK).max(axis=2) / MAX, MIN_SCALE)


def quantise(v):
    s = scales(v)
    return encode(v / np.repeat(s, BLOCK, axis=1)[:, :v.shape[1]]), s


def rmsnorm(x, residual, weight, eps):
    """-> (v, n) in float64."""
    v = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    r = 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    return v, v * r * np.asarray(weight, np.float64)


def gemm(a, w):
    """-> (A W^T, |A| |W|^T): the product and the sum of its terms' magnitudes."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def grouped(a, mats, offsets, entries, a_div):
    """Bucket-ordered products of every expert's rows: (y, magnitudes) of
    [n_pairs, N]; positions of no bucket are NaN."""
    P, N = len(entries), mats.shape[1]
    y, m = np.full((P, N), np.nan), np.full((P, N), np.nan)
    for e in range(mats.shape[0]):
        p = np.arange(offsets[e], offsets[e + 1])
        if len(p):
            src = np.asarray(entries)[p] // a_div if a_div > 0 else p
            y[p], m[p] = gemm(a[src], mats[e])
    return y, m
