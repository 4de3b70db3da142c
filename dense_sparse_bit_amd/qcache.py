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

from .qgemv import _check, _launch, lib as _qgemv_lib


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
        import torch
        self.n_pages, self.n_heads, self.head_dim = int(n_pages), int(n_heads), int(head_dim)
        self.page_size, self.group = int(page_size), int(group)
        n = cache_bytes(self.n_pages, self.n_heads, self.head_dim, self.page_size, self.group)
        self.data = torch.empty(n, dtype=torch.uint8, device=device)
        self._shape = Shape(self.n_pages, self.n_heads, self.head_dim, self.page_size, self.group)

    def _seqs(self, lens, pages, q_start, n_tok):
        import torch
        dev, i32 = self.data.device, torch.int32
        if lens.dtype != i32 or lens.dim() != 1 or not lens.is_contiguous():
            raise ValueError("lens must be a contiguous int32 [S] tensor")
        S = lens.shape[0]
        if pages.dtype != i32 or pages.dim() != 2 or pages.shape[0] != S or not pages.is_contiguous():
            raise ValueError("pages must be a contiguous int32 [S, P] tensor")
        if lens.device != dev or pages.device != dev:
            raise ValueError(f"all tensors must be on the cache's device {dev}")
        start = None
        if q_start is not None:
            if q_start.dtype != i32 or tuple(q_start.shape) != (S + 1,) or not q_start.is_contiguous():
                raise ValueError("q_start must be a contiguous int32 [S + 1] tensor")
            if q_start.device != dev:
                raise ValueError(f"all tensors must be on the cache's device {dev}")
            start = q_start.data_ptr()
        elif n_tok != S:
            raise ValueError("without q_start there is one row per sequence")
        return Seqs(S, n_tok, pages.shape[1], start, lens.data_ptr(), pages.data_ptr())

    def _rows(self, t, heads, what, types):
        """A [T, heads, head_dim] tensor as the library takes it; where a stride does not matter it is 0."""
        if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != self.head_dim or t.dtype not in types:
            raise ValueError(f"{what} must be a [T, {heads}, {self.head_dim}] tensor of {types}")
        ts, hs, ds = t.stride()
        if ds != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
        if t.device != self.data.device:
            raise ValueError(f"all tensors must be on the cache's device {self.data.device}")
        return Rows(t.data_ptr(), 0 if t.element_size() == 2 else 1, ts if t.shape[0] > 1 else 0,
                    hs if heads > 1 else 0)

    def write(self, k, v, lens, pages, q_start=None, stream=None):
        """Quantise the rows of k and v [T, n_heads, head_dim] (both FP16 or both fp32) into their positions.

        k and v may be views with strides that are multiples of 8 elements (columns of a stacked q/k/v
        product), starting on 16 bytes.
        """
        import torch
        if v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must have the same shape and type")
        types = (torch.float16, torch.float32)
        kr, vr = self._rows(k, self.n_heads, "k", types), self._rows(v, self.n_heads, "v", types)
        sq = self._seqs(lens, pages, q_start, k.shape[0])
        with _launch(self.data.device, stream) as s:
            _check(lib().qcache_write(self._shape, self.data.data_ptr(), sq, kr, vr, s), "qcache_write")

    def read(self, lens, pages, q_start=None, n_tok=None, k=None, v=None, dtype=None, stream=None):
        """(k, v): the values held where write() would have put the rows, [n_tok, n_heads, head_dim].

        Allocated as dtype (FP16 by default) if k and v are not given; rows of padding are then not
        initialised.  n_tok: rows of the outputs, by default those of k, or one per sequence.
        """
        import torch
        types = (torch.float16, torch.float32)
        if (k is None) != (v is None):
            raise ValueError("give both k and v, or neither")
        if n_tok is None:
            n_tok = k.shape[0] if k is not None else lens.shape[0]
            if k is None and q_start is not None:
                raise ValueError("with q_start the number of rows must be given: n_tok, or k and v")
        if dtype is not None and (dtype not in types or (k is not None and k.dtype != dtype)):
            raise ValueError("dtype must be torch.float16 or torch.float32, and that of k and v")
        if k is not None and (k.shape != v.shape or k.dtype != v.dtype or k.shape[0] != n_tok):
            raise ValueError("k and v must have the same shape and type, and n_tok rows")
        sq = self._seqs(lens, pages, q_start, n_tok)
        with _launch(self.data.device, stream) as s:
            if k is None:
                shape = (n_tok, self.n_heads, self.head_dim)
                k = torch.empty(shape, dtype=dtype or types[0], device=self.data.device)
                v = torch.empty(shape, dtype=dtype or types[0], device=self.data.device)
            kr, vr = self._rows(k, self.n_heads, "k", types), self._rows(v, self.n_heads, "v", types)
            _check(lib().qcache_read(self._shape, self.data.data_ptr(), sq, kr, vr, s), "qcache_read")
        return k, v

    def attend(self, q, lens, pages, q_start=None, scale=None, out=None, stream=None):
        """Attention of the rows of q [T, q_heads, head_dim] (FP16) over the cache, each up to its own position.

        q_heads is a multiple of n_heads; query head h reads key/value head h // (q_heads // n_heads).
        scale: 1 / sqrt(head_dim) by default.  out: FP16, the shape of q, allocated if not given (rows of
        padding are then not initialised); it must not overlap q.  A row that sees nothing is 0.
        """
        import torch
        if q.dim() != 3 or q.shape[1] < 1 or q.shape[1] % self.n_heads:
            raise ValueError(f"q must be [T, heads, {self.head_dim}] with a multiple of {self.n_heads} heads")
        H = q.shape[1]
        qr = self._rows(q, H, "q", (torch.float16,))
        sq = self._seqs(lens, pages, q_start, q.shape[0])
        scale = 1.0 / math.sqrt(self.head_dim) if scale is None else float(scale)
        if not math.isfinite(scale):
            raise ValueError("scale must be finite")
        if out is not None and out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        n = ctypes.c_size_t(0)
        _check(lib().qcache_attend_ws(self._shape, sq, H, n), "qcache_attend_ws")
        with _launch(self.data.device, stream) as s:
            if out is None:
                out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
            orow = self._rows(out, H, "out", (torch.float16,))
            ws = torch.empty(n.value, dtype=torch.uint8, device=q.device)
            _check(lib().qcache_attend(self._shape, self.data.data_ptr(), sq, H, qr, orow, scale, ws.data_ptr(),
                                       n.value, s), "qcache_attend")
        return out
