"""ctypes binding of the rotation by position fused with the cache's writing (include/qrotary.h).

As in qgemv.py, the arithmetic runs in the library's HIP kernels; PyTorch owns
the memory and names the stream, and there is no fallback.
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import qcache
from .qgemv import QgemvError, _launch, _stream_here, lib as _qgemv_lib

STYLE = {"halves": 0, "neighbours": 1}


class _Rotary(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("style", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("freqs", ctypes.c_void_p), ("pair_axis", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """The library with the C signature of include/qrotary.h declared."""
    global _lib
    if _lib is None:
        L = _qgemv_lib()
        P, vp = ctypes.POINTER, ctypes.c_void_p
        L.qrotary_write.argtypes = [P(qcache.Shape), vp, P(qcache.Seqs), P(_Rotary), ctypes.c_int32, P(qcache.Rows),
                                    P(qcache.Rows), P(qcache.Rows), P(qcache.Rows), vp]
        L.qrotary_write.restype = ctypes.c_int
        _lib = L
    return _lib


def _on(a, dtype, device):
    if isinstance(a, torch.Tensor):
        return a.to(device=device, dtype=dtype).contiguous()
    return torch.from_numpy(np.array(a, dtype={torch.float64: np.float64, torch.int32: np.int32}[dtype])).to(device)


class Rotary:
    """The turn of a head's first 2 * len(freqs) dimensions by position.

    freqs: radians per position of each pair (64 bits), for instance base ** (-2 i / rot_dim), scaled as the model has
    it.  style: "halves" (pair i = dimensions i and rot_dim / 2 + i) or "neighbours" (2 i and 2 i + 1).
    pair_axis: for positions of several axes (time, height, width), the axis by which each pair turns; a pair with an
    axis that positions do not have is left as it is.
    """

    def __init__(self, freqs, style="halves", pair_axis=None, device="cuda"):
        if style not in STYLE:
            raise ValueError(f"style must be one of {sorted(STYLE)}")
        if isinstance(freqs, torch.Tensor) and freqs.is_cuda:
            device = freqs.device
        self.freqs = _on(freqs, torch.float64, device)
        if self.freqs.dim() != 1:
            raise ValueError("freqs must be one-dimensional")
        self.rot_dim, self.style = 2 * self.freqs.shape[0], style
        self.pair_axis = None if pair_axis is None else _on(pair_axis, torch.int32, self.freqs.device)
        if self.pair_axis is not None and self.pair_axis.shape != self.freqs.shape:
            raise ValueError("pair_axis must have an axis for each of freqs")

    def write(self, cache, q, k, v, lens, pages, q_start=None, positions=None, out=None, stream=None):
        """Turns the rows of q [T, q_heads, head_dim] and k [T, n_heads, head_dim], writes k and v into the cache
        (QCache.write), and returns the turned q.

        positions: int32 [T] or [axes, T]; by default a row's own position in its sequence.  Where a row is stored
        goes by lens, pages and q_start in either case.  q: FP16 or fp32, or None (keys and values only).  out: FP16 or
        fp32 in the shape of q, q itself allowed; FP16 if not given, rows of padding then not initialised.
        """
        at = cache.data.get_device()
        s = _stream_here(at, stream)
        if s is None:
            with _launch(at, stream):
                return self.write(cache, q, k, v, lens, pages, q_start, positions, out)
        if self.freqs.get_device() != at:
            raise ValueError("the rotation must be on the cache's device")
        if k.dim() != 3 or v.dim() != 3:
            raise ValueError("k and v must be [T, heads, head_dim]")
        kr, vr = cache._rows(k, cache.n_heads, "k", at), cache._rows(v, cache.n_heads, "v", at)
        T = k.shape[0]
        if v.shape[0] != T or kr.type != vr.type:
            raise ValueError("k and v must have the same shape and type")
        sq = cache._seqs(lens, pages, q_start, T, at)
        axes, pos = 1, None
        if positions is not None:
            if positions.dim() == 1:
                positions = positions.unsqueeze(0)
            axes = positions.shape[0]
            if positions.dtype != torch.int32 or positions.shape != (axes, T) or not positions.is_contiguous() or (
                    positions.get_device() != at):
                raise ValueError("positions must be a contiguous int32 [T] or [axes, T] tensor on the cache's device")
            pos = positions.data_ptr()
        ro = _Rotary(self.rot_dim, STYLE[self.style], axes, self.freqs.data_ptr(),
                     None if self.pair_axis is None else self.pair_axis.data_ptr(), pos)
        H, qr, orow = 0, None, None
        if q is not None:
            if q.dim() != 3 or q.shape[0] != T:
                raise ValueError("q must be [T, heads, head_dim] with k's rows")
            H = q.shape[1]
            qr = cache._rows(q, H, "q", at)
            if out is None:
                D = cache.head_dim
                out = q.new_empty(T, H, D, dtype=torch.float16)
                orow = qcache.Rows(out.data_ptr(), 0, H * D, D)
            else:
                if out.shape != q.shape:
                    raise ValueError("out must be in the shape of q")
                orow = cache._rows(out, H, "out", at, True)
        elif out is not None:
            raise ValueError("out needs q")
        st = lib().qrotary_write(cache._shape, cache.data.data_ptr(), sq, ro, H, qr, orow, kr, vr, s)
        if st != 0:
            raise QgemvError(st, "qrotary_write")
        return out
