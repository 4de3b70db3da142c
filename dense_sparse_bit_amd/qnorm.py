"""ctypes binding of the norms around a block, fused with gate and residual stream (include/qnorm.h).

As in qgemv.py, the arithmetic runs in the library's HIP kernels; PyTorch owns
the memory and names the stream, and there is no fallback.
"""

from __future__ import annotations

import ctypes
import math

import torch

from .qgemv import QgemvError, _launch, _stream_here, lib as _qgemv_lib
from .qmx import FORMAT, MxRows

KIND = {"rms": 0, "layer": 1}
_BLOCKS = 16  # type of an output in MX blocks: this plus the format
_TYPE = {"fp16": torch.float16, "fp32": torch.float32}


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("type", ctypes.c_int32), ("ld", ctypes.c_int64)]


class Args(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("kind", ctypes.c_int32), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float)] + [(n, Rows) for n in ("y", "h", "gate", "post", "post_bias", "pre",
                                                                  "pre_bias", "h_out", "out")]


_lib = None


def lib() -> ctypes.CDLL:
    """The library with the C signature of include/qnorm.h declared."""
    global _lib
    if _lib is None:
        L = _qgemv_lib()
        L.qnorm_run.argtypes = [ctypes.POINTER(Args), ctypes.c_void_p]
        L.qnorm_run.restype = ctypes.c_int
        _lib = L
    return _lib


def _matrix(t, T, N, at, what):
    dt = t.dtype
    if (dt != torch.float16 and dt != torch.float32) or t.shape != (T, N) or t.get_device() != at:
        raise ValueError(f"{what} must be an FP16 or fp32 [T, N] tensor on the same device")
    ld, one = t.stride()
    if one != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return Rows(t.data_ptr(), dt == torch.float32, ld if T > 1 else 0)


def _vector(t, N, at, what):
    dt = t.dtype
    if (dt != torch.float16 and dt != torch.float32) or t.shape != (N,) or not t.is_contiguous() or t.get_device() != at:
        raise ValueError(f"{what} must be a contiguous FP16 or fp32 [N] tensor on the same device")
    return Rows(t.data_ptr(), dt == torch.float32, 0)


def norm(y, h=None, post=None, post_bias=None, gate=None, scale=1.0, pre=None, pre_bias=None, kind="rms", eps=1e-6,
         h_out=None, out=None, out_type="fp16", keep_h=True, stream=None):
    """The norms after and before a block, with the gate and the residual stream between them; returns (h', out).

        b   = y, or norm(y) * post + post_bias
        h'  = scale * h + gate * b
        out = norm(h') * pre + pre_bias

    y [T, N]: what the block computed, or None (the first norm of a model: h' = scale * h); h [T, N]: the residual stream,
    or None.  post, post_bias, pre, pre_bias: [N]; gate: [N] or [T, N].  All FP16 or fp32, rows of wider arrays
    allowed, on one GPU.  Without pre there is no out (None).  kind: "rms" (the mean square) or "layer" (mean and
    variance).  h' has h's type (y's without h); h_out: a tensor to write it into, h or y itself allowed; with keep_h False it is
    not written (None).  out_type: "fp16", "fp32", or "e2m1" / "e4m3" for MxRows, which QMx.run takes; out: what to
    write into, a tensor (h or y itself allowed) or MxRows, in place of out_type.
    """
    lead = y if y is not None else h
    if lead is None:
        raise ValueError("y or h must be given")
    at = lead.get_device()
    s = _stream_here(at, stream)
    if s is None:
        with _launch(at, stream):
            return norm(y, h, post, post_bias, gate, scale, pre, pre_bias, kind, eps, h_out, out, out_type, keep_h)
    if lead.dim() != 2:
        raise ValueError("y and h must be [T, N]")
    if kind not in KIND:
        raise ValueError(f"kind must be one of {sorted(KIND)}")
    if not (math.isfinite(eps) and eps >= 0 and math.isfinite(scale)):
        raise ValueError("eps must be finite and not negative, scale finite")
    T, N = lead.shape
    if max(T, N) > 2**31 - 1:
        raise ValueError("counts are 32-bit")
    a = Args(T, N, KIND[kind], eps, scale)
    if y is not None:
        a.y = _matrix(y, T, N, at, "y")
    if h is not None:
        a.h = _matrix(h, T, N, at, "h")
    if gate is not None:
        if y is None:
            raise ValueError("a gate needs y")
        a.gate = _vector(gate, N, at, "gate") if gate.dim() == 1 else _matrix(gate, T, N, at, "gate")
    for name, v in (("post", post), ("post_bias", post_bias), ("pre", pre), ("pre_bias", pre_bias)):
        if v is not None:
            setattr(a, name, _vector(v, N, at, name))
    if (post is None and post_bias is not None) or (pre is None and pre_bias is not None) or (y is None and post is not None):
        raise ValueError("a bias needs its weight, and post needs y")
    if h_out is None and keep_h:
        h_out = torch.empty_like(h if h is not None else y, memory_format=torch.contiguous_format)
    if h_out is not None:
        a.h_out = _matrix(h_out, T, N, at, "h_out")
    if pre is None:
        if out is not None:
            raise ValueError("out needs pre")
        if h_out is None:
            raise ValueError("there is nothing to write")
    else:
        if out is None:
            if out_type in FORMAT:
                out = MxRows(T, N, out_type, lead.device)
            elif out_type in _TYPE:
                out = lead.new_empty(T, N, dtype=_TYPE[out_type])
            else:
                raise ValueError(f"out_type must be one of {sorted([*_TYPE, *FORMAT])}")
        if isinstance(out, MxRows):
            if (out.rows, out.cols) != (T, N) or out.data.get_device() != at:
                raise ValueError("out must be [T, N] on the same device")
            a.out = Rows(out.data.data_ptr(), _BLOCKS + FORMAT[out.fmt], 0)
        else:
            a.out = _matrix(out, T, N, at, "out")
    if T > 0:
        st = lib().qnorm_run(a, s)
        if st != 0:
            raise QgemvError(st, "qnorm_run")
    return h_out, out
