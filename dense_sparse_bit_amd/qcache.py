"""ctypes binding of the 4-bit key/value cache and its attention (include/qcache.h).

As in qgemv.py, the arithmetic runs in the library's HIP kernels; PyTorch owns
the memory and names the stream, and there is no fallback.

Every call describes its batch the same way:

lens     int32 [S]: tokens of each sequence, the call's own rows included
pages    int32 [S, P]: page of each page_size positions; ids outside the pool hold nothing
q_start  int32 [S + 1], or None for one row per sequence: sequence s owns the
         rows q_start[s] .. q_start[s + 1] - 1 of k, v, q and the outputs, and row i
         of its n stands at position lens[s] - n + i.  Rows behind the last
         sequence's are padding and are left as they were.

They are read on the GPU when the kernels run, so a captured call follows
their contents.
"""

from __future__ import annotations

import ctypes
import math

import torch

from .qgemv import QgemvError, _check, _launch, _stream_here, lib as _qgemv_lib


_MAX = 2**31 - 1


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_pages", "n_heads", "head_dim", "page_size", "group")]


class Seqs(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_tok", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("q_start", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("pages", ctypes.c_void_p)]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("type", ctypes.c_int32), ("tok_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The library with the cache's C signatures declared."""
    global _lib
    if _lib is None:
        L = _qgemv_lib()
        P, vp = ctypes.POINTER, ctypes.c_void_p
        L.qcache_bytes.argtypes = [P(Shape), P(ctypes.c_size_t)]
        L.qcache_write.argtypes = [P(Shape), vp, P(Seqs), P(Rows), P(Rows), vp]
        L.qcache_read.argtypes = [P(Shape), vp, P(Seqs), P(Rows), P(Rows), vp]
        L.qcache_attend_ws.argtypes = [P(Shape), P(Seqs), ctypes.c_int32, P(ctypes.c_size_t)]
        L.qcache_attend.argtypes = [P(Shape), vp, P(Seqs), ctypes.c_int32, P(Rows), P(Rows), ctypes.c_float, vp,
                                    ctypes.c_size_t, vp]
        for f in ("qcache_bytes", "qcache_write", "qcache_read", "qcache_attend_ws", "qcache_attend"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def cache_bytes(n_pages, n_heads, head_dim, page_size=64, group=32) -> int:
    """Bytes of a cache of that shape."""
    if max(n_pages, n_heads, head_dim, page_size, group) > _MAX:
        raise ValueError("counts are 32-bit")
    n = ctypes.c_size_t(0)
    _check(lib().qcache_bytes(ctypes.byref(Shape(n_pages, n_heads, head_dim, page_size, group)), ctypes.byref(n)),
           "qcache_bytes")
    return n.value


class QCache:
    """A cache of n_pages pages of page_size tokens for n_heads key/value heads, in 4 bits.

    head_dim 64, 128 or 256; page_size a power of two, 16 .. 1024; group (dimensions that share a step and a
    lowest value) 32, 64 or 128.  data is its memory; a page holds nothing of use until it is written.
    """

    def __init__(self, n_pages, n_heads, head_dim, page_size=64, group=32, device="cuda"):
        self.n_pages, self.n_heads, self.head_dim = int(n_pages), int(n_heads), int(head_dim)
        self.page_size, self.group = int(page_size), int(group)
        n = cache_bytes(self.n_pages, self.n_heads, self.head_dim, self.page_size, self.group)
        self.data = torch.empty(n, dtype=torch.uint8, device=device)
        self._shape = Shape(self.n_pages, self.n_heads, self.head_dim, self.page_size, self.group)

    def _seqs(self, lens, pages, q_start, n_tok, at):
        i32 = torch.int32
        S = lens.shape[0]
        if lens.dtype != i32 or lens.shape != (S,) or not lens.is_contiguous() or lens.get_device() != at:
            raise ValueError("lens must be a contiguous int32 [S] tensor on the cache's device")
        P = pages.shape[-1]
        if pages.dtype != i32 or pages.shape != (S, P) or not pages.is_contiguous() or pages.get_device() != at:
            raise ValueError("pages must be a contiguous int32 [S, P] tensor on the cache's device")
        if S > _MAX or P > _MAX or n_tok > _MAX:
            raise ValueError("counts are 32-bit")
        if q_start is None:
            if n_tok != S:
                raise ValueError("without q_start there is one row per sequence")
            return Seqs(S, n_tok, P, None, lens.data_ptr(), pages.data_ptr())
        if q_start.dtype != i32 or q_start.shape != (S + 1,) or not q_start.is_contiguous() or (
                q_start.get_device() != at):
            raise ValueError("q_start must be a contiguous int32 [S + 1] tensor on the cache's device")
        return Seqs(S, n_tok, P, q_start.data_ptr(), lens.data_ptr(), pages.data_ptr())

    def _rows(self, t, heads, what, at, written=False):
        """A [T, heads, head_dim] tensor as the library takes it; a stride that does not matter is 0."""
        dt, T = t.dtype, t.shape[0]
        if (dt != torch.float16 and dt != torch.float32) or t.shape != (T, heads, self.head_dim) or (
                t.get_device() != at):
            raise ValueError(f"{what} must be an FP16 or fp32 [T, {heads}, {self.head_dim}] tensor on the cache's device")
        ts, hs, one = t.stride()
        if one != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
        if written:
            span = self.head_dim
            for stride, n in sorted(((ts, T), (hs, heads))):
                if n > 1 and stride < span:
                    raise ValueError(f"{what}: vectors must not overlap")
                if n > 1:
                    span += stride * (n - 1)
        return Rows(t.data_ptr(), dt == torch.float32, ts if T > 1 else 0, hs if heads > 1 else 0)

    def write(self, k, v, lens, pages, q_start=None, stream=None):
        """Quantise the rows of k and v [T, n_heads, head_dim] (both FP16 or both fp32) into their positions.

        k and v may be views with strides that are multiples of 8 elements (columns of a stacked q/k/v
        product), starting on 16 bytes.
        """
        at = self.data.get_device()
        s = _stream_here(at, stream)
        if s is None:
            with _launch(at, stream):
                return self.write(k, v, lens, pages, q_start)
        kr, vr = self._rows(k, self.n_heads, "k", at), self._rows(v, self.n_heads, "v", at)
        if v.shape[0] != k.shape[0] or kr.type != vr.type:
            raise ValueError("k and v must have the same shape and type")
        sq = self._seqs(lens, pages, q_start, k.shape[0], at)
        st = lib().qcache_write(self._shape, self.data.data_ptr(), sq, kr, vr, s)
        if st != 0:
            raise QgemvError(st, "qcache_write")

    def read(self, lens, pages, q_start=None, n_tok=None, k=None, v=None, dtype=None, stream=None):
        """(k, v): the values held where write() would have put the rows, [n_tok, n_heads, head_dim].

        Allocated as dtype (FP16 by default) if k and v are not given; rows of padding are then not
        initialised.  k and v, if given, must not overlap each other.  n_tok: rows of the outputs, by default those of k, or one per sequence.
        """
        at = self.data.get_device()
        s = _stream_here(at, stream)
        if s is None:
            with _launch(at, stream):
                return self.read(lens, pages, q_start, n_tok, k, v, dtype)
        if k is None and v is None:
            if n_tok is None:
                if q_start is not None:
                    raise ValueError("with q_start the number of rows must be given: n_tok, or k and v")
                n_tok = lens.shape[0]
            if dtype is None:
                dtype = torch.float16
            elif dtype != torch.float16 and dtype != torch.float32:
                raise ValueError("dtype must be torch.float16 or torch.float32")
            H, D = self.n_heads, self.head_dim
            k, v = self.data.new_empty(2, n_tok, H, D, dtype=dtype).unbind(0)
            kr, vr = (Rows(t.data_ptr(), dtype == torch.float32, H * D, D) for t in (k, v))
        elif k is None or v is None:
            raise ValueError("give both k and v, or neither")
        else:
            kr, vr = self._rows(k, self.n_heads, "k", at, True), self._rows(v, self.n_heads, "v", at, True)
            if v.shape[0] != k.shape[0] or kr.type != vr.type or n_tok not in (None, k.shape[0]):
                raise ValueError("k and v must have the same shape and type, and n_tok rows")
            if dtype is not None and dtype != k.dtype:
                raise ValueError("dtype is not that of k and v")
            n_tok = k.shape[0]
        sq = self._seqs(lens, pages, q_start, n_tok, at)
        st = lib().qcache_read(self._shape, self.data.data_ptr(), sq, kr, vr, s)
        if st != 0:
            raise QgemvError(st, "qcache_read")
        return k, v

    def attend(self, q, lens, pages, q_start=None, scale=None, out=None, stream=None):
        """Attention of the rows of q [T, q_heads, head_dim] (FP16) over the cache, each up to its own position.

        q_heads is a multiple of n_heads; query head h reads key/value head h // (q_heads // n_heads).
        scale: 1 / sqrt(head_dim) by default.  out: FP16, the shape of q, allocated if not given (rows of
        padding are then not initialised); it must not overlap q.  A row that sees nothing is 0.
        """
        at = self.data.get_device()
        s = _stream_here(at, stream)
        if s is None:
            with _launch(at, stream):
                return self.attend(q, lens, pages, q_start, scale, out)
        if q.dim() != 3 or q.shape[1] < 1 or q.shape[1] % self.n_heads or q.dtype != torch.float16:
            raise ValueError(f"q must be FP16 [T, heads, {self.head_dim}] with a multiple of {self.n_heads} heads")
        T, H = q.shape[0], q.shape[1]
        qr = self._rows(q, H, "q", at)
        sq = self._seqs(lens, pages, q_start, T, at)
        if scale is None:
            scale = 1.0 / math.sqrt(self.head_dim)
        elif not math.isfinite(scale):
            raise ValueError("scale must be finite")
        if out is None:
            out = q.new_empty(T, H, self.head_dim)
            orow = Rows(out.data_ptr(), 0, H * self.head_dim, self.head_dim)
        else:
            if out.shape != q.shape or out.dtype != torch.float16:
                raise ValueError("out must be FP16 in the shape of q")
            orow = self._rows(out, H, "out", at, True)
        n = ctypes.c_size_t(0)
        L = lib()
        st = L.qcache_attend_ws(self._shape, sq, H, n)
        if st == 0:
            # its own for every call: calls on other streams, and captured ones, never share it
            ws = self.data.new_empty(n.value)
            st = L.qcache_attend(self._shape, self.data.data_ptr(), sq, H, qr, orow, scale, ws.data_ptr(), n.value, s)
        if st != 0:
            raise QgemvError(st, "qcache_attend")
        return out
