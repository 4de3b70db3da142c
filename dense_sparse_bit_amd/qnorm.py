"""ctypes binding of the norms around a block, fused with gate and residual stream (include/qnorm.h).

As in qgemv.py, the arithmetic runs in the library's HIP kernels; PyTorch owns
the memory and names the stream, and there is no fallback.
"""

from __future__ import annotations

import ctypes
import math
import struct

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


# an Args' bytes from plain numbers in one step
_args = struct.Struct("@iiiff" + 9 * "Piq").pack
_NONE = (0, 0, 0)

_lib = None


def lib() -> ctypes.CDLL:
    """The library with the C signature of include/qnorm.h declared."""
    global _lib
    if _lib is None:
        L = _qgemv_lib()
        L.qnorm_run.argtypes = [ctypes.c_void_p, ctypes.c_void_p]  # an Args by reference, or its bytes
        L.qnorm_run.restype = ctypes.c_int
        _lib = L
    return _lib


def _matrix(t, T, N, at, what):
    """(pointer, is fp32, row stride) of a [T, N] tensor with contiguous rows; a stride that does not matter is 0."""
    f32 = t.dtype is torch.float32
    if (not f32 and t.dtype is not torch.float16) or t.shape != (T, N) or t.get_device() != at:
        raise ValueError(f"{what} must be an FP16 or fp32 [T, N] tensor on the same device")
    ld, one = t.stride()
    if one != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.data_ptr(), f32, ld if T > 1 else 0


def _vector(t, N, at, what):
    f32 = t.dtype is torch.float32
    if (not f32 and t.dtype is not torch.float16) or t.shape != (N,) or t.stride(0) != 1 or t.get_device() != at:
        raise ValueError(f"{what} must be a contiguous FP16 or fp32 [N] tensor on the same device")
    return t.data_ptr(), f32, 0


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
    if (post is None and post_bias is not None) or (pre is None and pre_bias is not None):
        raise ValueError("a bias needs its weight")
    if y is None and (gate is not None or post is not None):
        raise ValueError("gate and post need y")
    a_y = _NONE if y is None else _matrix(y, T, N, at, "y")
    a_h = _NONE if h is None else _matrix(h, T, N, at, "h")
    a_gate = _NONE if gate is None else _vector(gate, N, at, "gate") if gate.dim() == 1 else _matrix(gate, T, N, at, "gate")
    a_post = _NONE if post is None else _vector(post, N, at, "post")
    a_pb = _NONE if post_bias is None else _vector(post_bias, N, at, "post_bias")
    a_pre = _NONE if pre is None else _vector(pre, N, at, "pre")
    a_prb = _NONE if pre_bias is None else _vector(pre_bias, N, at, "pre_bias")
    a_ho = a_out = _NONE
    if h_out is not None:
        a_ho = _matrix(h_out, T, N, at, "h_out")
    elif keep_h:
        like = y if h is None else h
        h_out = like.new_empty(T, N)
        a_ho = (h_out.data_ptr(), like.dtype is torch.float32, N)
    if pre is None:
        if out is not None:
            raise ValueError("out needs pre")
        if h_out is None:
            raise ValueError("there is nothing to write")
    elif out is None and out_type in _TYPE:
        out = lead.new_empty(T, N, dtype=_TYPE[out_type])
        a_out = (out.data_ptr(), out_type == "fp32", N)
    else:
        if out is None:
            if out_type not in FORMAT:
                raise ValueError(f"out_type must be one of {sorted([*_TYPE, *FORMAT])}")
            out = MxRows(T, N, out_type, lead.device)
        if isinstance(out, MxRows):
            if out.rows != T or out.cols != N or out.data.get_device() != at:
                raise ValueError("out must be [T, N] on the same device")
            a_out = (out.data.data_ptr(), _BLOCKS + FORMAT[out.fmt], 0)
        else:
            a_out = _matrix(out, T, N, at, "out")
    if T > 0:
        st = lib().qnorm_run(_args(T, N, KIND[kind], eps, scale, *a_y, *a_h, *a_gate, *a_post, *a_pb, *a_pre, *a_prb, *a_ho,
                                   *a_out), s)
        if st != 0:
            raise QgemvError(st, "qnorm_run")
    return h_out, out
