"""Oracle of rows in microscaled blocks and of their product, in fp64 numpy -- test infrastructure only.

Storage (include/qmx.h): blocks of 32 columns with one power of two 2^(b - 127)
and elements on the grid of E2M1 or E4M3.  A quantised element is the grid point
nearest to value / 2^(b - 127), the even code where two are as near; b is the
smallest byte whose grid reaches the block's largest value, or with clip the
one that puts the largest value's binade on the grid's last; 1 at least.
"""

from __future__ import annotations

import math

import numpy as np


def grid(fmt: str) -> np.ndarray:
    """Magnitudes by code, from 0 up."""
    if fmt == "e2m1":
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
    g = [(8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9 for e in range(16) for m in range(8)]
    return np.array(g[:-1], dtype=np.float64)  # the last code is NaN


def quantise(x, fmt: str, clip: bool = False):
    """x [T, K] -> (codes uint8 [T, K] with the sign in the top bit of 4 or 8, exponent bytes uint8 [T, K / 32])."""
    g = grid(fmt)
    x = np.asarray(x).astype(np.float64)
    T, K = x.shape
    b = x.reshape(T, K // 32, 32)
    codes = np.zeros(b.shape, dtype=np.uint8)
    exps = np.zeros(b.shape[:2], dtype=np.uint8)
    sign = 8 if fmt == "e2m1" else 128
    for t in range(T):
        for i in range(K // 32):
            v = b[t, i]
            if not np.isfinite(v).all():
                exps[t, i] = 255
                continue
            top = np.abs(v).max()
            e = -126
            if top > 0:
                if clip:
                    e = math.frexp(top)[1] - math.frexp(g[-1])[1]
                else:
                    e = math.frexp(top)[1] - 12
                    while top > g[-1] * 2.0 ** e:
                        e += 1
            e = max(e, -126)
            exps[t, i] = e + 127
            a = np.minimum(np.abs(v) / 2.0 ** e, g[-1])
            hi = np.searchsorted(g, a)
            lo = np.maximum(hi - 1, 0)
            up, down = g[hi] - a, a - g[lo]
            c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            codes[t, i] = c + np.where(np.signbit(v), sign, 0)
    return codes.reshape(T, K), exps


def values(codes, exps, fmt: str) -> np.ndarray:
    g = grid(fmt)
    sign = 8 if fmt == "e2m1" else 128
    c = np.asarray(codes).astype(np.int64)
    m = c & (sign - 1)
    v = np.where(m < len(g), g[np.minimum(m, len(g) - 1)], np.nan) * np.where(c & sign, -1.0, 1.0)
    step = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127))
    return v * np.repeat(step, 32, axis=1)


def pack_bytes(codes, fmt: str) -> np.ndarray:
    """Codes as the plain arrays hold them: two E2M1 codes a byte, the lower column below."""
    codes = np.asarray(codes, dtype=np.uint8)
    return codes if fmt == "e4m3" else codes[:, 0::2] | (codes[:, 1::2] << 4)


def activate(t, act: str):
    if act == "relu":
        return np.maximum(t, 0)
    if act == "silu":
        return t * np.exp(-np.logaddexp(0, -t))
    if act == "gelu":
        return t * np.vectorize(lambda z: 0.5 * math.erfc(-z / math.sqrt(2)))(t)
    if act == "gelu_tanh":
        return t * np.exp(-np.logaddexp(0, -math.sqrt(8 / math.pi) * (t + 0.044715 * t ** 3)))
    return t


def product(x, w, bias=None, act="none", gated=False, residual=None):
    """(y, tol): the product of values x [T, K] and w [M, K] with its epilogue, and how far fp32 sums may leave it.

    The products of two elements are exact, so a sum of K of them in chunks of 128 is off by at most
    (128 + K / 128 + 16) 2^-24 of the sum of magnitudes A, one rounding more for the bias.  The activations' slopes are
    at most 1.13, they are formed to 8 ulps, and a gated pair's errors add up by the product rule.
    """
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    t = x @ w.T
    A = np.abs(x) @ np.abs(w).T
    if bias is not None:
        t = t + np.asarray(bias, np.float64)
        A = A + np.abs(np.asarray(bias, np.float64))
    d = (128 + x.shape[1] / 128 + 16) * 2.0 ** -24 * A + 2.0 ** -126
    if gated:
        g, u = t[:, 0::2], t[:, 1::2]
        a = activate(g, act)
        da = 1.13 * d[:, 0::2] + 2.0 ** -20 * np.abs(a)
        y = a * u
        d = np.abs(a) * d[:, 1::2] + np.abs(u) * da + da * d[:, 1::2] + 2.0 ** -24 * np.abs(y)
    else:
        y = activate(t, act)
        d = 1.13 * d + 2.0 ** -20 * np.abs(y)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
        d = d + 2.0 ** -24 * np.abs(y)
    return y, d
