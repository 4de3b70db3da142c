"""ctypes binding of rows in microscaled blocks and their product (include/qmx.h).

As in qgemv.py, the arithmetic runs in the library's HIP kernels; PyTorch owns
the memory and names the stream, and there is no fallback.

A block is 32 neighbouring columns of a row: elements in 4 bits ("e2m1") or 8
("e4m3"), and a power of two that they share.
"""

from __future__ import annotations

import ctypes

import torch

from .qgemv import ACT, Epilogue, QGemv, QgemvError, _check, _launch, _stream_here, lib as _qgemv_lib

FORMAT = {"e2m1": 0, "e4m3": 1}
_IN_BLOCKS = -1
_MAX = 2**31 - 1


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "cols", "format")]


class Input(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int32), ("format", ctypes.c_int32),
                ("x_type", ctypes.c_int32), ("ldx", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The library with the C signatures of include/qmx.h declared."""
    global _lib
    if _lib is None:
        L = _qgemv_lib()
        P, vp, i32, sz = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.qmx_bytes.argtypes = [P(Shape), P(sz)]
        L.qmx_quantize.argtypes = [P(Shape), vp, vp, i32, ctypes.c_int64, i32, vp]
        L.qmx_values.argtypes = [P(Shape), vp, vp, i32, ctypes.c_int64, vp]
        L.qmx_pack.argtypes = [P(Shape), vp, vp, vp, vp]
        L.qmx_unpack.argtypes = [P(Shape), vp, vp, vp, vp]
        L.qmx_run_ws.argtypes = [P(Shape), P(Input), P(Epilogue), P(sz)]
        L.qmx_run.argtypes = [P(Shape), vp, P(Input), vp, P(Epilogue), vp, sz, vp]
        for f in ("qmx_bytes", "qmx_quantize", "qmx_values", "qmx_pack", "qmx_unpack", "qmx_run_ws", "qmx_run"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _format(fmt):
    if fmt not in FORMAT:
        raise ValueError(f"the format must be one of {sorted(FORMAT)}")
    return FORMAT[fmt]


def _rows(x, what, at=None):
    """(is fp32, row stride) of an FP16 or fp32 [T, K] tensor with contiguous rows; a stride that does not matter is 0."""
    f32 = x.dtype is torch.float32
    strides = x.stride()
    if (not f32 and x.dtype is not torch.float16) or len(strides) != 2 or (at is not None and x.get_device() != at):
        raise ValueError(f"{what} must be an FP16 or fp32 [T, K] tensor" + ("" if at is None else " on the same device"))
    if strides[1] != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return f32, strides[0] if len(x) > 1 else 0


class MxRows:
    """Rows [rows, cols] in MX blocks; data is their memory, in the library's own order."""

    def __init__(self, rows, cols, fmt="e2m1", device="cuda"):
        if rows > _MAX or cols > _MAX:
            raise ValueError("counts are 32-bit")
        self.rows, self.cols, self.fmt = int(rows), int(cols), fmt
        self._shape = Shape(self.rows, self.cols, _format(fmt))
        n = ctypes.c_size_t(0)
        st = lib().qmx_bytes(self._shape, n)
        if st != 0:
            raise QgemvError(st, "qmx_bytes")
        self.data = torch.empty(n.value, dtype=torch.uint8, device=device)

    @classmethod
    def pack(cls, codes, exponents, fmt="e2m1", stream=None):
        """From plain arrays on the GPU: codes uint8 [rows, cols / 2], the lower column in the lower nibble (e2m1), or
        [rows, cols] (e4m3), and exponents uint8 [rows, cols / 32]: powers of two 2^(b - 127)."""
        at = codes.get_device()
        if _stream_here(at, stream) is None:
            with _launch(at, stream):
                return cls.pack(codes, exponents, fmt)
        _format(fmt)
        if codes.dim() != 2 or codes.dtype != torch.uint8 or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous uint8 [rows, bytes] tensor")
        rows, cols = codes.shape[0], codes.shape[1] * (2 if fmt == "e2m1" else 1)
        if exponents.dtype != torch.uint8 or exponents.shape != (rows, cols // 32) or not exponents.is_contiguous() or (
                exponents.get_device() != at):
            raise ValueError("exponents must be a contiguous uint8 [rows, cols / 32] tensor on the same device")
        out = cls(rows, cols, fmt, codes.device)
        _check(lib().qmx_pack(out._shape, out.data.data_ptr(), codes.data_ptr(), exponents.data_ptr(),
                              _stream_here(at, None)), "qmx_pack")
        return out

    def unpack(self, stream=None):
        """(codes, exponents) as pack() takes them."""
        at = self.data.get_device()
        s = _stream_here(at, stream)
        if s is None:
            with _launch(at, stream):
                return self.unpack()
        codes = self.data.new_empty(self.rows, self.cols // (2 if self.fmt == "e2m1" else 1))
        exponents = self.data.new_empty(self.rows, self.cols // 32)
        _check(lib().qmx_unpack(self._shape, self.data.data_ptr(), codes.data_ptr(), exponents.data_ptr(), s), "qmx_unpack")
        return codes, exponents

    def values(self, dtype=torch.float32, out=None, stream=None):
        """The values that the blocks stand for, [rows, cols], FP16 or fp32 (rounded once)."""
        at = self.data.get_device()
        s = _stream_here(at, stream)
        if s is None:
            with _launch(at, stream):
                return self.values(dtype, out)
        if out is None:
            f32, ld = dtype is torch.float32, self.cols
            if not f32 and dtype is not torch.float16:
                raise ValueError("dtype must be torch.float16 or torch.float32")
            out = self.data.new_empty(self.rows, ld, dtype=dtype)
        else:
            if out.shape != (self.rows, self.cols):
                raise ValueError("out must be [rows, cols]")
            f32, ld = _rows(out, "out", at)
        st = lib().qmx_values(self._shape, self.data.data_ptr(), out.data_ptr(), f32, ld, s)
        if st != 0:
            raise QgemvError(st, "qmx_values")
        return out


def quantize(x, fmt="e2m1", clip=False, out=None, stream=None):
    """x [T, K] (FP16 or fp32 on the GPU, K a multiple of 32, rows of a wider array allowed) in MX blocks.

    The block's power of two is the smallest that reaches its largest value; with clip, the largest value's own less
    the element's, so that values above the largest element are held at it.  out: MxRows to write into.
    """
    at = x.get_device()
    s = _stream_here(at, stream)
    if s is None:
        with _launch(at, stream):
            return quantize(x, fmt, clip, out)
    f32, ld = _rows(x, "x")
    T, K = x.shape
    if out is None:
        out = MxRows(T, K, fmt, x.device)
    elif out.rows != T or out.cols != K or out.fmt != fmt or out.data.get_device() != at:
        raise ValueError("out must have x's shape, the format, and be on x's device")
    st = lib().qmx_quantize(out._shape, out.data.data_ptr(), x.data_ptr(), f32, ld, bool(clip), s)
    if st != 0:
        raise QgemvError(st, "qmx_quantize")
    return out


class QMx:
    """A weight set [M, K] in E2M1 blocks (MxRows, for instance quantize(w) or MxRows.pack) and its products."""

    def __init__(self, w: MxRows):
        if w.fmt != "e2m1":
            raise ValueError("weights are in the format e2m1")
        self.w, self.M, self.K = w, w.rows, w.cols

    def run(self, x, x_fmt="e2m1", bias=None, act="none", gated=False, residual=None, out=None, dtype=None, stream=None):
        """act(x W^T + bias) + residual, or with gated (rows 2i, 2i + 1 of W = gate, up) act(gate) * up + residual;
        returns out [T, M] ([T, M // 2] gated).

        x: MxRows [T, K], or FP16 or fp32 [T, K], which are quantised to x_fmt on the way; any T.  bias [M] and
        residual [T, M or M // 2]: FP16 or fp32.  act: "none", "relu", "gelu", "gelu_tanh" or "silu".  out: FP16 or
        fp32, allocated as dtype (FP16 by default) if not given; out and residual may be rows of wider arrays, and
        residual may be out itself; out overlaps nothing else that the call reads.  All on the weights' device.
        """
        at = self.w.data.get_device()
        s = _stream_here(at, stream)
        if s is None:
            with _launch(at, stream):
                return self.run(x, x_fmt, bias, act, gated, residual, out, dtype)
        if isinstance(x, MxRows):
            T = x.rows
            if x.cols != self.K or x.data.get_device() != at:
                raise ValueError("x must have the weights' columns and be on their device")
            xi = Input(x.data.data_ptr(), T, FORMAT[x.fmt], _IN_BLOCKS, 0)
        else:
            if x.dim() == 1:
                x = x.unsqueeze(0)
            f32, ld = _rows(x, "x", at)
            T = x.shape[0]
            if x.shape[1] != self.K or T > _MAX:
                raise ValueError("x must have the weights' columns")
            xi = Input(x.data_ptr(), T, _format(x_fmt), f32, ld)
        if act not in ACT:
            raise ValueError(f"act must be one of {sorted(ACT)}")
        mo = self.M // 2 if gated else self.M
        e = Epilogue(ACT[act], bool(gated))
        if bias is not None:
            f32 = bias.dtype == torch.float32
            if (not f32 and bias.dtype != torch.float16) or bias.shape != (self.M,) or not bias.is_contiguous() or (
                    bias.get_device() != at):
                raise ValueError("bias must be a contiguous FP16 or fp32 [M] tensor on the weights' device")
            e.bias, e.bias_type = bias.data_ptr(), f32
        if residual is not None:
            e.residual, e.residual_type, e.ldr = QGemv._output_rows(residual, T, mo, at, "residual")
        if out is None:
            if dtype is None:
                dtype = torch.float16
            elif dtype != torch.float16 and dtype != torch.float32:
                raise ValueError("dtype must be torch.float16 or torch.float32")
            out = self.w.data.new_empty(T, mo, dtype=dtype)
            y, e.y_type = out.data_ptr(), dtype == torch.float32
        else:
            if dtype is not None and dtype != out.dtype:
                raise ValueError("dtype is not that of out")
            y, e.y_type, e.ldy = QGemv._output_rows(out, T, mo, at, "out")
        L, ws, size = lib(), None, 0
        if not isinstance(x, MxRows):  # blocks need none
            n = ctypes.c_size_t(0)
            _check(L.qmx_run_ws(self.w._shape, xi, e, n), "qmx_run_ws")
            size = n.value
            if size:
                # its own for every call: calls on other streams, and captured ones, never share it
                ws = self.w.data.new_empty(size)
        st = L.qmx_run(self.w._shape, self.w.data.data_ptr(), xi, y, e, ws.data_ptr() if size else None, size, s)
        if st != 0:
            raise QgemvError(st, "qmx_run")
        return out
