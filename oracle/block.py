"""Oracle of the norms around a block and of the rotation by position, in fp64 numpy -- test infrastructure only."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32


def unit(x, dx, weight, bias, kind, eps):
    """norm(x) * weight + bias, and how far fp32 may leave it where x is off by dx already.

    Sums of n values run over at most 64 values a lane, 6 exchanges and 16 waves: 96 roundings.  Squares are positive,
    so their sum is off by 96 U of itself, its root by half that, division and root by U each; a mean is off by 96 U of
    the mean magnitude.
    """
    mean, dm = 0.0, 0.0
    if kind == "layer":
        mean = x.mean(axis=1, keepdims=True)
        dm = dx.mean(axis=1, keepdims=True) + 98 * U * np.abs(x).mean(axis=1, keepdims=True)
    c = x - mean
    dc = dx + dm + U * np.abs(c)
    s = np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
    ds = np.sqrt((dc * dc).mean(axis=1, keepdims=True)) / s + 52 * U
    u = c / s
    y = u * weight
    dy = np.abs(weight) * (dc / s + np.abs(u) * ds) + 3 * U * np.abs(y)
    if bias is not None:
        y = y + bias
        dy = dy + U * np.abs(y)
    return y, dy


def norm(y, h=None, post=None, post_bias=None, gate=None, scale=1.0, pre=None, pre_bias=None, kind="rms", eps=1e-6):
    """((h', tolerance), (out, tolerance)) of include/qnorm.h, before the roundings to the outputs' types."""
    f = lambda a: None if a is None else np.asarray(a, dtype=np.float64)  # noqa: E731
    y, h, post, post_bias, gate, pre, pre_bias = map(f, (y, h, post, post_bias, gate, pre, pre_bias))
    scale, eps = float(np.float32(scale)), float(np.float32(eps))
    b = np.zeros_like(h) if y is None else y
    db = np.zeros_like(b)
    if post is not None:
        b, db = unit(b, db, post, post_bias, kind, eps)
    if gate is not None:
        b, db = gate * b, np.abs(gate) * db + U * np.abs(gate * b)
    if h is not None:
        db = db + U * (np.abs(scale * h) + np.abs(scale * h + b))
        b = scale * h + b
    return (b, db), (None if pre is None else unit(b, db, pre, pre_bias, kind, eps))


def turned(x, positions, freqs, style: str, pair_axis=None):
    """x [T, H, D] with its first 2 * len(freqs) dimensions turned by positions [axes, T], fp64."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    positions = np.asarray(positions)
    for i, f in enumerate(np.asarray(freqs, dtype=np.float64)):
        ax = 0 if pair_axis is None else int(pair_axis[i])
        if not 0 <= ax < len(positions):
            continue
        # the product of the position and the frequency is fp64 by definition; long double for what follows it
        a = (positions[ax].astype(np.float64) * f).astype(np.longdouble)
        c, s = (np.asarray(g(a), dtype=np.float64)[:, None] for g in (np.cos, np.sin))
        p, q = (i, len(freqs) + i) if style == "halves" else (2 * i, 2 * i + 1)
        out[..., p] = x[..., p] * c - x[..., q] * s
        out[..., q] = x[..., q] * c + x[..., p] * s
    return out
