"""Oracle of the 4-bit key/value cache and of attention over it, in fp64 numpy -- test infrastructure only.

Storage (include/qcache.h): values are rounded to FP16; a group of `group`
dimensions keeps lo = min, s = fp16((max - lo) / 15) and codes
q = clamp(rint((v - lo) / s), 0, 15).  The difference, the quotients and rint are
FP32 by definition, so they are FP32 here; everything after them is fp64.
"""

from __future__ import annotations

import numpy as np


def quantise(v, group: int):
    """v [..., D] -> dict of q (uint8 [..., D]), s and lo (FP16 [..., D / group])."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        x = np.asarray(v).astype(np.float16).astype(np.float32)
        x = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
        bad = ~np.isfinite(x).all(axis=-1)
        lo = x.min(axis=-1)
        s = ((x.max(axis=-1) - lo) / np.float32(15)).astype(np.float16)
        top = lo + np.float32(15) * s.astype(np.float32)
        s = np.where(top > 65504, np.nextafter(s, np.float16(0)), s)
        r = np.rint((x - lo[..., None]) / s.astype(np.float32)[..., None])
        q = np.where((s[..., None] > 0) & ~bad[..., None], np.clip(r, 0, 15), 0)
        q = np.nan_to_num(q).astype(np.uint8)
    s = np.where(bad, np.float16(np.nan), s).astype(np.float16)
    lo = np.where(bad, np.float32(0), lo).astype(np.float16)
    return {"q": q.reshape(np.asarray(v).shape), "s": s, "lo": lo}


def values(enc: dict) -> np.ndarray:
    """lo + s q in fp64 (exact)."""
    q = enc["q"].astype(np.float64)
    g = q.shape[-1] // enc["s"].shape[-1]
    q = q.reshape(q.shape[:-1] + (enc["s"].shape[-1], g))
    out = enc["lo"].astype(np.float64)[..., None] + enc["s"].astype(np.float64)[..., None] * q
    return out.reshape(enc["q"].shape)


def held(v, group: int) -> np.ndarray:
    """The values that the cache holds for v, fp64."""
    return values(quantise(v, group))


def reach(enc: dict) -> np.ndarray:
    """|lo| + 15 s of every value's group: bounds each part of the value."""
    g = enc["q"].shape[-1] // enc["s"].shape[-1]
    b = np.abs(enc["lo"].astype(np.float64)) + 15 * enc["s"].astype(np.float64)
    return np.repeat(b, g, axis=-1)


def attend(q, k, v, scale: float, last, mask=None):
    """softmax(scale q k^T) v of one sequence.

    q [n, Hq, D]; k, v [L, H, D] fp64 (held values); row i sees the positions
    p <= last[i] (and mask[p], if given).  Returns out [n, Hq, D] and the mean
    of |v| under the weights, [n, Hq, D]; rows that see nothing are 0.
    """
    q = np.asarray(q, dtype=np.float64)
    n, Hq, D = q.shape
    L, H, _ = k.shape
    per = Hq // H
    out, mean = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for i in range(n):
        see = np.arange(L) <= last[i]
        if mask is not None:
            see &= mask
        if not see.any():
            continue
        for h in range(Hq):
            s = scale * (k[see, h // per] @ q[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ v[see, h // per]
            mean[i, h] = p @ np.abs(v[see, h // per])
    return out, mean
