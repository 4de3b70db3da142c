"""The 4-bit key/value cache (qcache_write, qcache_read) and attention over it
(qcache_attend) against the fp64 oracle.

Write and read: the storage is defined to the bit, so what is read back in
fp32 must equal fp32(lo + s q) (one FP32 rounding of an exact value), and in
FP16 its rounding.

Attention, per output element, with E = the mean of |v| under the weights:
  weights   rounded to FP16: 2^-11 of each (2^-25 absolute below 2^-14, where
            the running maximum leaves the largest weight at 1 or more: n 2^-25
            of the largest |v| in all); so is each value: 2^-11
  scores    fp32 sums of exact products: off by at most 2^-18 of
            scale sum |q| (|lo| + 15 s) =: B (64 roundings of 2^-24), and the
            difference to the maximum is rounded, 2^-23 of |S| <= B; exp2 adds 2^-22:
            a weight is off by a factor 1 + (2^-18 + 2^-23) B + 2^-22, numerator
            and denominator each
  sums      fp32: (n / 32 + 16) 2^-24 each
  output    2^-11 of the value, 2^-25 where it is subnormal
"""

import ctypes
import math
import re

import numpy as np
import pytest

from dense_sparse_bit_amd import qcache, qgemv
from gpu_checks import say
from oracle import cache as oc


# ---------------------------------------------------------------------------
# CPU
# ---------------------------------------------------------------------------
def test_library_exports_every_declared_symbol():
    with open(qgemv.HEADER.replace("qgemv.h", "qcache.h")) as f:
        names = set(re.findall(r"^int (qcache_\w+)\(", f.read(), re.M))
    assert names == {"qcache_bytes", "qcache_write", "qcache_read", "qcache_attend_ws", "qcache_attend"}
    for n in names:
        assert hasattr(qcache.lib(), n), n


@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_cache_bytes(D, G, page):
    # 4 bits a value and 4 bytes a group, keys and values
    assert qcache.cache_bytes(7, 3, D, page, G) == 7 * 3 * page * 2 * (D // 2 + 4 * (D // G))


@pytest.mark.parametrize("shape,want", [
    ((0, 1, 128, 64, 32), -1), ((-3, 1, 128, 64, 32), -1), ((1, 0, 128, 64, 32), -1), ((1, 65536, 128, 64, 32), -3),
    ((1, 1, 96, 64, 32), -3), ((1, 1, 0, 64, 32), -3), ((1, 1, 128, 48, 32), -3), ((1, 1, 128, 8, 32), -3),
    ((1, 1, 128, 2048, 32), -3), ((1, 1, 128, 64, 16), -3), ((1, 1, 64, 64, 128), -3), ((1, 1, 128, 64, 0), -3)])
def test_shapes_refused(shape, want):
    n = ctypes.c_size_t(0)
    assert qcache.lib().qcache_bytes(ctypes.byref(qcache.Shape(*shape)), ctypes.byref(n)) == want


def test_calls_refused_on_the_host():
    """Everything that is refused before a launch; the pointers are never followed."""
    L, sh = qcache.lib(), qcache.Shape(4, 2, 128, 64, 32)
    ok = dict(n_seq=2, n_tok=2, max_pages=1, q_start=None, lens=4096, pages=4096)
    rows = qcache.Rows(4096, 0, 256, 128)

    def sq(**kw):
        return qcache.Seqs(*{**ok, **kw}.values())

    def copy(f, sh=sh, cache=4096, seqs=None, k=rows, v=rows):
        return f(ctypes.byref(sh), cache, seqs or sq(), k, v, None)

    for f in (L.qcache_write, L.qcache_read):
        assert copy(f, sh=qcache.Shape(4, 2, 100, 64, 32)) == -3
        assert copy(f, cache=None) == -1 and copy(f, cache=4096 + 128) == -1
        assert f(ctypes.byref(sh), 4096, None, rows, rows, None) == -1
        assert f(ctypes.byref(sh), 4096, sq(), None, rows, None) == -1
        assert copy(f, seqs=sq(n_seq=-1)) == -1 and copy(f, seqs=sq(n_tok=-1)) == -1
        assert copy(f, seqs=sq(max_pages=-1)) == -1 and copy(f, seqs=sq(max_pages=1 << 25)) == -3
        assert copy(f, seqs=sq(n_tok=3)) == -1  # no q_start
        assert copy(f, seqs=sq(lens=None)) == -1 and copy(f, seqs=sq(pages=None)) == -1
        assert copy(f, seqs=sq(lens=4098)) == -1 and copy(f, seqs=sq(q_start=4097, n_tok=3)) == -1
        for bad, want in [((None, 0, 256, 128), -1), ((4104, 0, 256, 128), -1), ((4096, 2, 256, 128), -3),
                          ((4096, 0, 252, 128), -1), ((4096, 0, 256, 4), -1)]:
            assert copy(f, k=qcache.Rows(*bad)) == want and copy(f, v=qcache.Rows(*bad)) == want
        assert copy(f, v=qcache.Rows(4096, 1, 256, 128)) == -1  # types differ
        assert copy(f, seqs=sq(n_seq=0, n_tok=0, lens=None, pages=None)) == 0
        assert copy(f, seqs=sq(n_tok=0)) == 0

    def att(sh=sh, cache=4096, seqs=None, heads=4, q=rows, out=rows, scale=1.0, ws=4096, n=1 << 30):
        return L.qcache_attend(ctypes.byref(sh), cache, seqs or sq(), heads, q, out, scale, ws, n, None)

    assert att(heads=0) == -1 and att(heads=3) == -3 and att(heads=65538) == -3
    assert att(scale=math.inf) == -1 and att(scale=math.nan) == -1
    assert att(cache=None) == -1 and att(ws=None) == -1 and att(ws=4096 + 16) == -1 and att(n=64) == -5
    assert att(q=qcache.Rows(4096, 1, 256, 128)) == -3 and att(out=qcache.Rows(4096, 1, 256, 128)) == -3
    assert att(q=qcache.Rows(4098, 0, 256, 128)) == -1 and att(seqs=sq(n_tok=3)) == -1
    # 2^31 blocks of 128 tokens
    assert att(seqs=sq(n_seq=1 << 20, n_tok=1 << 20, max_pages=1 << 12)) == -3
    assert att(seqs=sq(n_seq=0, n_tok=0, lens=None, pages=None)) == 0
    n = ctypes.c_size_t(0)
    assert L.qcache_attend_ws(ctypes.byref(sh), sq(), 3, n) == -3
    assert L.qcache_attend_ws(ctypes.byref(sh), sq(), 4, None) == -1
    assert L.qcache_attend_ws(ctypes.byref(sh), sq(), 4, n) == 0 and 0 < n.value < 1 << 26


def test_oracle_quantiser():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal((50, 64)) * 10.0 ** rng.integers(-6, 4, (50, 1)),
                        np.zeros((1, 64)), np.full((1, 64), -3.25), np.full((1, 64), 65504.0)])
    v16 = v.astype(np.float16).astype(np.float64)
    e = oc.quantise(v, 32)
    step = np.repeat(e["s"].astype(np.float64), 32, axis=-1)
    # half a step, 15/2 of the step's own rounding (2^-11 of it, 2^-25 where it is subnormal), and the quotient's FP32
    assert np.all(np.abs(oc.values(e) - v16) <= step * (0.5 + 2.0 ** -20) + 15 * (step * 2.0 ** -11 + 2.0 ** -25))
    assert np.array_equal(oc.values(e)[-3:], v16[-3:])  # constant groups are exact
    assert (e["q"].reshape(-1, 32).min(axis=1) == 0).all()
    w = v.copy()
    w[0, 3], w[1, 40], w[2, 0] = np.inf, np.nan, 1e6
    h = oc.held(w, 32)
    assert np.isnan(h[0, :32]).all() and np.isnan(h[1, 32:]).all() and np.isnan(h[2, :32]).all()
    assert np.isfinite(h[0, 32:]).all() and np.isfinite(h[3:]).all()
    # the widest group: the step is lowered so that no held value passes FP16's range
    wide = np.concatenate([np.full((1, 31), -65504.0), [[65504.0]]], axis=1)
    assert np.abs(oc.held(wide, 32)).max() <= 65504


def test_oracle_attention_by_hand():
    k = np.array([[[1.0, 0.0]], [[0.0, 2.0]], [[5.0, 5.0]]])
    v = np.array([[[1.0, 10.0]], [[3.0, -2.0]], [[100.0, 100.0]]])
    q = np.array([[[1.0, 1.0], [0.0, 0.0]]])
    out, mean = oc.attend(q, k, v, 0.5, [1])
    e = math.exp(0.5) / (math.exp(0.5) + math.exp(1.0))
    assert np.allclose(out[0, 0], [e + 3 * (1 - e), 10 * e - 2 * (1 - e)])
    assert np.allclose(out[0, 1], [2, 4]) and np.allclose(mean[0, 1], [2, 6])
    assert not oc.attend(q, k, v, 0.5, [-1])[0].any()
    assert np.allclose(oc.attend(q, k, v, 0.5, [2], np.array([True, False, False]))[0], v[0, 0])


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


class Batch:
    """Sequences of given lengths and new rows over shuffled pages; the arrays of the calls."""

    def __init__(self, torch, lens, new, page, pad=0, spare=2, seed=0, one_each=False):
        rng = np.random.default_rng(seed)
        need = [max(0, -(-n // page)) for n in lens]
        self.total = sum(need) + spare
        order = rng.permutation(self.total).astype(np.int32)
        self.table = np.full((len(lens), max(need + [1])), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.lens, self.new, self.page = list(lens), list(new), page
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n_tok = int(self.start[-1]) + pad
        cu = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        self.d_lens, self.d_pages = cu(self.lens), cu(self.table)
        self.d_start = None if one_each else cu(self.start)

    def args(self):
        return self.d_lens, self.d_pages, self.d_start

    def positions(self, s):
        n = self.new[s]
        return np.arange(max(self.lens[s], 0) - n, max(self.lens[s], 0))

    def on_page(self, s, pos):
        ok = (pos >= 0) & (pos < self.table.shape[1] * self.page)
        ok[ok] = (self.table[s, pos[ok] // self.page] >= 0) & (self.table[s, pos[ok] // self.page] < self.total)
        return ok


DIMS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def poison(torch, c):
    """A cache that was never written may hold anything: all bits set reads as NaN statistics."""
    c.data.fill_(0xFF)
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("D,G", DIMS)
@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_write_then_read(torch, D, G, dtype):
    """Ragged rows (none, one, many; more rows than positions), padding rows, a page missing, one out of the pool."""
    for page, H in ((16, 3), (64, 1), (256, 2)):
        b = Batch(torch, [70, 0, 1, 5, 333, 16, -4], [40, 2, 1, 9, 333, 0, 1], page, pad=3, seed=D + G + page)
        b.table[4, 0], b.table[0, 1 if page < 64 else 0] = -1, b.total + 5
        b.d_pages.copy_(torch.from_numpy(b.table))
        say(f"[gpu] cache write/read D={D} G={G} page={page} heads={H} {dtype}")
        rng = np.random.default_rng(D * G + page)
        kv = [(rng.standard_normal((b.n_tok, H, D)) * 10.0 ** rng.integers(-3, 3, (b.n_tok, H, 1))
               + rng.standard_normal((H, D))).astype(dtype) for _ in range(2)]
        c = poison(torch, qcache.QCache(b.total, H, D, page_size=page, group=G))
        c.write(*[torch.from_numpy(a).cuda() for a in kv], *b.args())
        for out in (torch.float32, torch.float16):
            mark = -12345.0
            got = [torch.full((b.n_tok, H, D), mark, dtype=out, device="cuda") for _ in range(2)]
            c.read(*b.args(), k=got[0], v=got[1])
            for g, a in zip(got, kv):
                want = np.full((b.n_tok, H, D), mark)
                with np.errstate(over="ignore"):
                    h = oc.held(a, G).astype(np.float32)
                for s in range(len(b.lens)):
                    ok = b.on_page(s, b.positions(s))
                    rows = slice(b.start[s], b.start[s + 1])
                    want[rows] = np.where(ok[:, None, None], h[rows], 0)
                want = want.astype(np.float32).astype(np.float16 if out == torch.float16 else np.float32)
                assert np.array_equal(g.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("n_seq", [63, 65, 130, 4099])
def test_write_many_sequences(torch, n_seq):
    """The search for a wave's sequence, one and two rounds of it; empty sequences and sequences without rows between."""
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, 40, n_seq).tolist()
    new = [int(min(n, k)) for n, k in zip(rng.integers(0, 35, n_seq), lens)]
    b = Batch(torch, lens, new, 16, pad=9, seed=n_seq)
    D, H = 64, 2
    k, v = (rng.standard_normal((b.n_tok, H, D)).astype(np.float16) for _ in range(2))
    say(f"[gpu] cache write, {n_seq} sequences")
    c = poison(torch, qcache.QCache(b.total, H, D, page_size=16, group=32))
    c.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), *b.args())
    got = c.read(*b.args(), n_tok=b.n_tok, dtype=torch.float32)
    for g, a in zip(got, (k, v)):
        assert np.array_equal(g.cpu().numpy()[:b.start[-1]], oc.held(a, 32).astype(np.float32)[:b.start[-1]])


@pytest.mark.gpu
@pytest.mark.parametrize("D,G", [(64, 32), (128, 128), (256, 64)])
def test_write_extremes(torch, D, G):
    rng = np.random.default_rng(5)
    T, H = 40, 2
    k = rng.standard_normal((T, H, D)).astype(np.float32)
    k[0] = 0
    k[1] = -3.25
    k[2, :, ::2], k[2, :, 1::2] = 65504, -65504
    k[3] = np.where(np.arange(D) % 3 == 0, 6e-8, 0)  # the smallest FP16 subnormal
    k[4] = rng.integers(-5, 6, (H, D)) * 2.0 ** -24
    k[5, 0, 7], k[6, 1, D - 1], k[7, 0, 0], k[8, 0, G - 1] = np.inf, np.nan, -np.inf, 7e4  # 7e4 is not finite in FP16
    k[9] = np.round(k[9] * 8) * 0.5  # many ties
    k[10] = rng.integers(0, 31, (H, D)) * 0.5
    k[11] = -0.0
    v = np.roll(k, 3, axis=0)
    b = Batch(torch, [T], [T], 16)
    say(f"[gpu] cache extremes D={D} G={G}")
    c = poison(torch, qcache.QCache(b.total, H, D, page_size=16, group=G))
    c.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), *b.args())
    got = c.read(*b.args(), n_tok=T, dtype=torch.float32)
    for g, a in zip(got, (k, v)):
        assert np.array_equal(g.cpu().numpy(), oc.held(a, G).astype(np.float32), equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,page", [(64, 64, 16), (128, 32, 64), (256, 128, 128)])
def test_write_leaves_other_tokens_alone(torch, D, G, page):
    """Every byte outside the written tokens keeps its value, and a step overwrites only its own position."""
    H, L = 3, 90
    b = Batch(torch, [L, L], [L, L], page, seed=1)
    rng = np.random.default_rng(2)
    mk = lambda n: torch.from_numpy(rng.standard_normal((n, H, D)).astype(np.float16)).cuda()
    c = poison(torch, qcache.QCache(b.total, H, D, page_size=page, group=G))
    k, v = mk(2 * L), mk(2 * L)
    c.write(k, v, *b.args())
    before, raw = c.read(*b.args(), n_tok=2 * L, dtype=torch.float32), c.data.clone()
    one = Batch(torch, [38, 0], [1, 1], page, one_each=True)
    k2, v2 = mk(2), mk(2)
    say(f"[gpu] cache step over a full cache D={D}")
    c.write(k2, v2, one.d_lens, b.d_pages)
    after = c.read(*b.args(), n_tok=2 * L, dtype=torch.float32)
    for x, y, new in zip(before, after, (k2, v2)):
        want = x.clone()
        want[37] = torch.from_numpy(oc.held(new[0].cpu().numpy(), G).astype(np.float32)).cuda()
        assert torch.equal(y, want)
    assert int((raw != c.data).sum()) <= H * 2 * (D // 2 + 4 * (D // G))


@pytest.mark.gpu
def test_strided_views_and_refusals(torch):
    """k and v as columns of a stacked q/k/v product, read back into columns of a wider array."""
    T, Hq, H, D = 21, 4, 2, 64
    qkv = torch.randn((T, (Hq + 2 * H) * D), device="cuda").half()
    k = qkv[:, Hq * D:(Hq + H) * D].view(T, H, D)
    v = qkv[:, (Hq + H) * D:].view(T, H, D)
    b = Batch(torch, [T], [T], 32)
    c = qcache.QCache(b.total, H, D, page_size=32, group=32)
    say("[gpu] cache strided views")
    c.write(k, v, *b.args())
    wide = torch.zeros((T, H, 2 * D + 8), device="cuda")
    kk, vv = c.read(*b.args(), k=wide[:, :, 8:8 + D], v=wide[:, :, 8 + D:])
    assert np.array_equal(kk.cpu().numpy(), oc.held(k.cpu().numpy(), 32).astype(np.float32))
    assert np.array_equal(vv.cpu().numpy(), oc.held(v.cpu().numpy(), 32).astype(np.float32))
    assert not wide[:, :, :8].any()
    kt = torch.randn((H, T, D), device="cuda").half().transpose(0, 1)  # head-major
    c.write(kt, kt, *b.args())
    assert np.array_equal(c.read(*b.args(), n_tok=T)[1].float().cpu().numpy(),
                          oc.held(kt.cpu().numpy(), 32).astype(np.float32).astype(np.float16).astype(np.float32))
    lens, pages, start = b.args()
    i64 = lens.long()
    for bad in (lambda: c.write(k, v.float(), lens, pages, start), lambda: c.write(k.bfloat16(), v.bfloat16(), lens, pages, start),
                lambda: c.write(k[:, :1], v[:, :1], lens, pages, start), lambda: c.write(k, v, lens, pages),
                lambda: c.write(k, v, i64, pages, start), lambda: c.write(k, v, lens, pages[0], start),
                lambda: c.write(k, v, lens, pages, start[:1]), lambda: c.write(k.cpu(), v.cpu(), lens, pages, start),
                lambda: c.write(k, v, lens.cpu(), pages, start),
                lambda: c.read(lens, pages, start), lambda: c.read(lens, pages, start, k=kk),
                lambda: c.read(lens, pages, start, n_tok=T, dtype=torch.int32),
                lambda: c.attend(qkv.view(T, -1, D)[:, :3], lens, pages, start),
                lambda: c.attend(k.float(), lens, pages, start), lambda: c.attend(k, lens, pages, start, scale=math.inf),
                lambda: c.attend(k, lens, pages, start, out=torch.zeros((T, H, D + 1), device="cuda").half())):
        with pytest.raises(ValueError):
            bad()
    flat = torch.zeros(T * H * D + 4, device="cuda").half()
    with pytest.raises(qgemv.QgemvError):  # 8 bytes off
        c.write(flat[4:].view(T, H, D), v, lens, pages, start)
    torch.cuda.synchronize()


def test_memory_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    c = qcache.QCache(2, 1, 64, page_size=16, device="cpu")
    lens, pages = torch.ones(1, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32)
    x = torch.zeros((1, 1, 64), dtype=torch.float16)
    for call in (lambda: c.write(x, x, lens, pages), lambda: c.read(lens, pages), lambda: c.attend(x, lens, pages)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("i", range(5))
def test_counts_past_32_bits(i):
    shape = [1, 1, 64, 64, 32]
    shape[i] += 2**32
    with pytest.raises(ValueError):
        qcache.cache_bytes(*shape)


def test_written_vectors_must_not_overlap():
    torch = pytest.importorskip("torch")
    T, H, D = 3, 2, 64
    c = qcache.QCache(1, H, D, device="cpu")
    x = torch.zeros(T * H * D + 64)
    wide = torch.zeros((T, H, 2 * D))
    for good in (x[:T * H * D].view(T, H, D), x[:T * H * D].view(H, T, D).transpose(0, 1), wide[:, :, D:],
                 x[:H * D].view(1, H, D), x[:0].view(0, H, D)):
        c._rows(good, H, "out", -1, True)
    for bad in (x[:H * D].view(1, H, D).expand(T, H, D), x[:T * D].view(T, 1, D).expand(T, H, D),
                x.as_strided((T, H, D), (H * D - 8, D, 1)), x.as_strided((T, H, D), (D, T * D - 8, 1)),
                x.as_strided((T, H, D), (D, D, 1)), x.as_strided((T, H, D), (H * D, D - 8, 1))):
        c._rows(bad, H, "k", -1)  # fine to read from
        with pytest.raises(ValueError):
            c._rows(bad, H, "out", -1, True)


@pytest.mark.gpu
def test_outputs_that_overlap_refused(torch):
    T, H, D = 5, 2, 64
    b = Batch(torch, [T], [T], 32)
    c = qcache.QCache(b.total, H, D, page_size=32)
    k = torch.randn((1, H, D), device="cuda").half().expand(T, H, D)  # one vector for every row may be written from
    c.write(k, k, *b.args())
    kk, vv = c.read(*b.args(), n_tok=T)
    assert np.array_equal(kk[3].cpu().numpy(), oc.held(k[:1].cpu().numpy(), 32).astype(np.float16)[0])
    with pytest.raises(ValueError):
        c.read(*b.args(), k=kk[:1].expand(T, H, D), v=vv)
    with pytest.raises(ValueError):
        c.attend(kk, *b.args(), out=vv[:1].expand(T, H, D))


# ---- attention ----------------------------------------------------------------
def fill(torch, b, H, D, G, seed, spread=1.0, keys=None, vals=None):
    """A cache holding every sequence of b whole; returns it and the held (encoded) keys and values."""
    rng = np.random.default_rng(seed)
    c = poison(torch, qcache.QCache(b.total, H, D, page_size=b.page, group=G))
    enc = []
    pos = [max(n, 0) for n in b.lens]
    for s, n in enumerate(pos):
        k = (rng.standard_normal((n, H, D)) * spread + rng.standard_normal((H, D))).astype(np.float16)
        v = rng.standard_normal((n, H, D)).astype(np.float16)
        if keys is not None:
            k = keys(s, k)
        if vals is not None:
            v = vals(s, v)
        enc.append((oc.quantise(k, G), oc.quantise(v, G)))
        if n:
            one = torch.tensor([n], dtype=torch.int32, device="cuda")
            st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            c.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), one, b.d_pages[s:s + 1].contiguous(), st)
    return c, enc


def check_attend(b, enc, q, got, scale, what, skip=()):
    g = got.float().cpu().numpy().astype(np.float64)
    worst = 0.0
    for s, (ek, ev) in enumerate(enc):
        n = b.new[s]
        if n == 0 or s in skip:
            continue
        L = ek["q"].shape[0]
        rows = slice(b.start[s], b.start[s + 1])
        qs = q[rows].astype(np.float64)
        pos = np.arange(L)
        mask = b.on_page(s, pos) if L else None
        k, v = oc.values(ek), oc.values(ev)
        want, mean = oc.attend(qs, k, v, scale, b.positions(s), mask)
        per = q.shape[1] // k.shape[1]
        if L:
            reach = oc.reach(ek)
            B = abs(scale) * np.stack([(np.abs(qs[:, h]) @ reach[:, h // per].T).max(axis=1) for h in range(q.shape[1])],
                                      axis=1)
            vmax = np.abs(v).max(axis=0)[np.arange(q.shape[1]) // per][None]
        else:
            B, vmax = np.zeros((n, q.shape[1])), 0.0
        rel = 2 * 2.0 ** -11 + 2 * ((2.0 ** -18 + 2.0 ** -23) * B + 2.0 ** -22)[..., None] + 2 * (L / 32 + 16) * 2.0 ** -24
        tol = rel * (mean + np.abs(want)) + L * 2.0 ** -25 * vmax
        tol = tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25
        err = np.abs(g[rows] - want)
        assert np.all(np.isfinite(g[rows])), f"{what}: sequence {s} is not finite"
        worst = max(worst, float((err / tol).max()))
        assert worst <= 1, f"{what}: sequence {s}, worst error {worst:.2f} of the tolerance"
    return worst


def queries(T, Hq, D, seed, size=1.0):
    return (np.random.default_rng(seed + 77).standard_normal((T, Hq, D)) * size).astype(np.float16)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G", DIMS)
@pytest.mark.parametrize("H,per", [(2, 1), (1, 4), (3, 7), (1, 8), (2, 16), (1, 20)])
def test_attend_one_row_each(torch, D, G, H, per):
    """Lengths around every border: none, one token, a unit, a tile, a block, a page."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 127, 128, 129, 161, 500]
    page = {64: 16, 128: 64, 256: 256}[D]
    b = Batch(torch, lens, [1] * len(lens), page, seed=G, one_each=True)
    c, enc = fill(torch, b, H, D, G, seed=D + per)
    q = queries(b.n_tok, H * per, D, seed=D)
    say(f"[gpu] attend D={D} G={G} heads={H} x {per}")
    out = torch.full((b.n_tok, H * per, D), float("nan"), dtype=torch.float16, device="cuda")
    got = c.attend(torch.from_numpy(q).cuda(), *b.args(), out=out)
    check_attend(b, enc, q, got, 1 / math.sqrt(D), f"D={D} G={G}")
    assert not got[0].any()  # the empty sequence
    assert torch.equal(got, c.attend(torch.from_numpy(q).cuda(), *b.args())), "not bitwise deterministic"


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,page", [(128, 32, 16), (64, 32, 128), (256, 128, 32)])
@pytest.mark.parametrize("H,per", [(1, 1), (2, 8), (2, 5)])
def test_attend_several_rows(torch, D, G, page, H, per):
    """Causal among the call's own rows; more rows than positions; no rows; padding rows keep their contents."""
    lens, new = [70, 3, 200, 16, 0, 140, 129], [5, 7, 1, 0, 2, 140, 33]
    b = Batch(torch, lens, new, page, pad=4, seed=3)
    c, enc = fill(torch, b, H, D, G, seed=per)
    q = queries(b.n_tok, H * per, D, seed=per)
    say(f"[gpu] attend rows D={D} G={G} heads={H} x {per} page={page}")
    mark = torch.full((b.n_tok, H * per, D), -7.5, dtype=torch.float16, device="cuda")
    got = c.attend(torch.from_numpy(q).cuda(), *b.args(), out=mark.clone())
    assert torch.equal(got[b.start[-1]:], mark[b.start[-1]:]), "padding rows were written"
    check_attend(b, enc, q, got, 1 / math.sqrt(D), f"rows D={D}")
    assert not got[5:9].any()  # rows in front of the first position


@pytest.mark.gpu
@pytest.mark.parametrize("n_seq", [63, 64, 65, 200])
def test_attend_many_sequences(torch, n_seq):
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, 300, n_seq).tolist()
    new = rng.integers(0, 3, n_seq).tolist()
    b = Batch(torch, lens, new, 16, seed=n_seq)
    c, enc = fill(torch, b, 2, 64, 32, seed=1)
    q = queries(b.n_tok, 4, 64, seed=n_seq)
    say(f"[gpu] attend {n_seq} sequences")
    check_attend(b, enc, q, c.attend(torch.from_numpy(q).cuda(), *b.args()), 0.125, f"{n_seq} sequences")


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,per", [([20011], 2, 2), ([9000, 1, 4096, 0, 17], 1, 8), ([70000], 1, 1)])
def test_attend_long(torch, lens, H, per):
    """Sequences that many workgroups share."""
    b = Batch(torch, lens, [1] * len(lens), 64, seed=1, one_each=True)
    c, enc = fill(torch, b, H, 128, 32, seed=9)
    q = queries(b.n_tok, H * per, 128, seed=5, size=2.0)
    say(f"[gpu] attend long {lens}")
    check_attend(b, enc, q, c.attend(torch.from_numpy(q).cuda(), *b.args()), 1 / math.sqrt(128), f"{lens}")


@pytest.mark.gpu
def test_attend_rising_and_falling_scores(torch):
    """The running maximum: scores that rise along the sequence, that fall, and a single far peak; small and
    large q (the scaling by powers of two), q with one huge element, zero q and a negative scale."""
    D, G, L = 128, 32, 1200
    ramp = np.linspace(-6, 6, L)[:, None, None]

    def keys(s, k):
        k = k * 0.1
        k[..., 0:1] = {0: ramp, 1: -ramp, 2: np.where(np.arange(L) == 700, 12.0, 0.0)[:, None, None], 3: ramp}[s]
        return k.astype(np.float16)

    b = Batch(torch, [L] * 4, [1] * 4, 64, seed=2, one_each=True)
    c, enc = fill(torch, b, 1, D, G, seed=4, keys=keys)
    for size, scale in ((1.0, 1.0), (3.0, 0.3), (1e-4, 500.0), (2000.0, 1e-4), (0.0, 1.0), (1.0, -1.0), (1.0, 0.0)):
        q = queries(4, 3, D, seed=8, size=0.2)
        q[:, 0, 0], q[:, 1, 0], q[:, 2, 0] = 4, -4, 1
        q = (q.astype(np.float64) * size).astype(np.float16)
        if size == 1.0:
            q[3, 2, 5] = 30000  # 2^20 and more above the others
        say(f"[gpu] attend ramps size={size} scale={scale}")
        check_attend(b, enc, q, c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=scale), scale, f"size {size} scale {scale}")


@pytest.mark.gpu
def test_attend_tiny_and_huge_values(torch):
    """Steps and values in FP16's subnormal range, and keys near its end; scales that bring the scores back."""
    D, G, L = 64, 32, 300
    b = Batch(torch, [L] * 4, [1] * 4, 64, seed=3, one_each=True)
    sizes = [(1e-5, 1e-5), (1e-6, 1.0), (3000.0, 3000.0), (1.0, 1e-6)]
    c, enc = fill(torch, b, 2, D, G, seed=6, keys=lambda s, k: (k.astype(np.float64) * sizes[s][0]).astype(np.float16),
                  vals=lambda s, v: (v.astype(np.float64) * sizes[s][1]).astype(np.float16))
    for size, scale in ((1.0, 0.125), (1.0, 1e4), (100.0, 1e-4)):
        q = queries(4, 4, D, seed=9, size=size)
        say(f"[gpu] attend tiny and huge values size={size} scale={scale}")
        got = c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=scale)
        # at 1e4 the scores of the last two sequences reach 1e8: fp32 sums are then off by whole units, so those two
        # are held only where the scores are small enough
        check_attend(b, enc, q, got, scale, f"scale {scale}", skip=(2, 3) if scale == 1e4 else ())
        assert torch.isfinite(got).all().item()
    # any finite scale: the largest score wins
    q = queries(4, 4, D, seed=9)
    got = c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=1e37)
    for s in (1, 3):
        k, v = oc.values(enc[s][0]), oc.values(enc[s][1])
        for h in range(4):
            best = np.sort(k[:, h // 2] @ q[s, h].astype(np.float64))
            if best[-1] - best[-2] > 1e-3 * best[-1]:
                want = v[np.argmax(k[:, h // 2] @ q[s, h].astype(np.float64)), h // 2]
                assert np.abs(got[s, h].float().cpu().numpy() - want).max() <= 2.0 ** -10 * np.abs(want).max() + 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("L,at", [(40000, 17), (40000, 39990), (5000, 2500)])
def test_attend_thin_tail(torch, L, at):
    """One position far above many whose values are large: each weight is 2^-26.5 of the largest, together they
    are most of the output.  A weight is held to half of FP16's least step, 2^-25, where the largest is 2^7 or
    more: to 2^-32 of it."""
    D, G = 64, 32
    tail = 400000.0 / L

    def keys(s, k):
        k = k * 0
        k[at, :, 0] = 1
        return k.astype(np.float16)

    def vals(s, v):
        v = v * 0.02 + tail
        v[at] = np.linspace(-0.01, 0.01, D)
        return v.astype(np.float16)

    b = Batch(torch, [L], [1], 64, seed=9, one_each=True)
    c, enc = fill(torch, b, 1, D, G, seed=6, keys=keys, vals=vals)
    q = np.zeros((1, 2, D), np.float16)
    q[:, :, 0] = 1
    scale = 26.5 * math.log(2)
    say(f"[gpu] attend thin tail L={L} at={at}")
    got = c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=scale)
    check_attend(b, enc, q, got, scale, "thin tail")
    k, v = (oc.values(e) for e in enc[0])
    want, mean = oc.attend(q.astype(np.float64), k, v, scale, b.positions(0), None)
    # values 2^-11, scores 2^-18 of 26.5 ln 2 in the exponent, sums (L / 32 + 16) 2^-24, and the weights as above
    rel = 2 * 2.0 ** -11 + 2 * 2.0 ** -18 * scale + (L / 32 + 16) * 2.0 ** -24
    tol = rel * (mean + np.abs(want)) + L * 2.0 ** -32 * np.abs(v).max() + 2.0 ** -25
    err = np.abs(got.float().cpu().numpy() - want)
    assert float((np.abs(want - v[at, 0]) / tol).min()) > 20  # the tail's part, which is what is looked at
    assert float((err / tol).max()) <= 1


@pytest.mark.gpu
def test_attend_nan_and_missing_pages(torch):
    """A NaN or infinite value counts exactly for the rows that see its token; pages that are no pages are
    masked; what lies behind a sequence's end (all bits set here) never shows."""
    D, G, H, per, page = 128, 32, 2, 4, 16
    lens, new = [100, 100, 100, 300], [6, 6, 6, 3]
    bad_k = lambda s, k: (k.__setitem__((97, 0, 5), np.nan), k)[1] if s == 1 else k
    bad_v = lambda s, v: (v.__setitem__((97, 1, 70), np.inf), v)[1] if s == 2 else v
    b = Batch(torch, lens, new, page, seed=6)
    b.table[3, [0, 4, 5, 18]] = [-1, b.total, 1 << 30, -(1 << 31)]  # the last page of sequence 3 too
    c, enc = fill(torch, b, H, D, G, seed=3, keys=bad_k, vals=bad_v)
    b.d_pages.copy_(torch.from_numpy(b.table))
    q = queries(b.n_tok, H * per, D, seed=1)
    q[1, 3, 7] = np.nan  # one row and head of sequence 0
    say("[gpu] attend NaN, infinities, missing pages")
    got = c.attend(torch.from_numpy(q).cuda(), *b.args())
    g = got.float().cpu().numpy()
    want_nan = np.zeros(g.shape, bool)
    want_nan[1, 3] = True
    # token 97 is seen by rows 3, 4, 5 (positions 97, 98, 99)
    want_nan[6 + 3:12, :per] = True
    want_nan[12 + 3:18, per:, 64:96] = True
    assert np.array_equal(np.isnan(g), want_nan)
    q2 = q.copy()
    q2[1, 3, 7] = 0
    clean = c.attend(torch.from_numpy(q2).cuda(), *b.args()).float().cpu().numpy()
    assert np.array_equal(clean[~want_nan], g[~want_nan])
    check_attend(b, enc, q2, torch.from_numpy(clean), 1 / math.sqrt(D), "missing pages", skip=(1, 2))
    # the rows of sequences 1 and 2 in front of token 97: as if the sequences ended there
    cut = Batch(torch, [97, 97], [3, 3], page)
    cut_enc = [tuple({key: a[:97] for key, a in e.items()} for e in enc[s]) for s in (1, 2)]
    rows = [6, 7, 8, 12, 13, 14]
    check_attend(cut, cut_enc, q2[rows], torch.from_numpy(clean[rows]), 1 / math.sqrt(D), "before the NaN")
    # a sequence whose every page is missing sees nothing
    none = torch.full_like(b.d_pages, -1)
    assert not c.attend(torch.from_numpy(q2).cuda(), b.d_lens, none, b.d_start).any()


@pytest.mark.gpu
def test_attend_table_shorter_than_the_lengths(torch):
    """Positions past the table hold nothing; a table with no pages at all."""
    b = Batch(torch, [200, 30], [2, 1], 16, seed=4)
    c, enc = fill(torch, b, 1, 64, 64, seed=2)
    q = queries(b.n_tok, 2, 64, seed=3)
    short = Batch(torch, [200, 30], [2, 1], 16, seed=4)
    short.table = short.table[:, :3]
    say("[gpu] attend with a short table")
    got = c.attend(torch.from_numpy(q).cuda(), b.d_lens, b.d_pages[:, :3].contiguous(), b.d_start)
    check_attend(short, enc, q, got, 0.125, "short table")
    empty = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    assert not c.attend(torch.from_numpy(q).cuda(), b.d_lens, empty, b.d_start).any()
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    nothing = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    assert c.attend(nothing, z, torch.empty((0, 3), dtype=torch.int32, device="cuda")).shape == (0, 2, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(24))
def test_random_calls(torch, seed):
    """Shapes, ragged and empty sequences, rows per sequence, padding, tables with holes, scales and output
    strides drawn together; attention twice (the same bits), and the cache read back in both types."""
    rng = np.random.default_rng(seed)
    D, G = DIMS[seed % len(DIMS)]
    H, per = int(rng.choice([1, 2, 3, 5])), int(rng.choice([1, 2, 3, 4, 7, 8, 17, 33]))
    page, S = int(rng.choice([16, 32, 64, 128, 1024])), int(rng.choice([1, 2, 3, 5, 9, 20]))
    top = int(np.exp(rng.uniform(0, math.log(5000 if S < 4 else 900))))
    lens = [int(rng.integers(0, top + 1)) if rng.random() < 0.9 else 0 for _ in range(S)]
    one_each = rng.random() < 0.4
    new = [1] * S if one_each else [int(rng.choice([0, 1, 1, 2, 3, 7, 17])) for _ in range(S)]
    b = Batch(torch, lens, new, page, pad=0 if one_each else int(rng.integers(1, 4)), seed=seed, one_each=one_each)
    c, enc = fill(torch, b, H, D, G, seed=seed, spread=float(rng.choice([0.2, 1, 3])))
    for _ in range(int(rng.integers(0, 5))):
        b.table[rng.integers(S), rng.integers(b.table.shape[1])] = [-1, b.total, 1 << 29][rng.integers(3)]
    b.d_pages.copy_(torch.from_numpy(b.table))
    scale = float(rng.choice([1 / math.sqrt(D), 1.0, 0.01, -0.1]))
    q = queries(b.n_tok, H * per, D, seed, float(rng.choice([1e-3, 0.3, 1, 4])))
    say(f"[gpu] random call {seed}: D={D} G={G} H={H} per={per} page={page} S={S} lens<={top} rows={b.n_tok}")
    end = int(b.start[-1])
    out = torch.full((b.n_tok, H * per, D + 8), 7.0, device="cuda").half()
    got = c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=scale, out=out[:, :, :D])
    check_attend(b, enc, q, got, scale, f"random call {seed}")
    assert bool((out[:, :, D:] == 7).all()) and bool((out[end:] == 7).all())
    again = c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=scale)
    assert torch.equal(again[:end], got[:end])
    for dtype in (torch.float16, torch.float32):
        wide = [torch.full((b.n_tok, H, D + 8), 3.0, device="cuda", dtype=dtype) for _ in range(2)]
        c.read(*b.args(), k=wide[0][:, :, :D], v=wide[1][:, :, :D])
        for i, w in enumerate(wide):
            assert bool((w[:, :, D:] == 3).all()) and bool((w[end:] == 3).all())
            for s in range(S):
                pos = b.positions(s)
                on = b.on_page(s, pos)
                want = np.zeros((len(pos), H, D))
                if on.any():
                    want[on] = oc.values(enc[s][i])[pos[on]]
                want = want.astype(np.float32)  # lo + s q in fp32, then the rows' type
                g = w[b.start[s]:b.start[s + 1], :, :D].cpu().numpy()
                assert np.array_equal(g, want if dtype == torch.float32 else want.astype(np.float16))


@pytest.mark.gpu
def test_attend_strided_q_and_out(torch):
    b = Batch(torch, [50, 333], [1, 1], 32, seed=1, one_each=True)
    c, enc = fill(torch, b, 2, 128, 64, seed=2)
    wide = torch.from_numpy(queries(2, 16, 128, seed=4)).cuda()
    q = wide[:, 3:11]
    out = torch.full((2, 8, 136), 3.0, dtype=torch.float16, device="cuda")
    say("[gpu] attend strided")
    got = c.attend(q, *b.args(), out=out[:, :, :128])
    check_attend(b, enc, q.cpu().numpy(), got, 1 / math.sqrt(128), "strided")
    assert torch.all(out[:, :, 128:] == 3.0)


@pytest.mark.gpu
def test_cache_past_four_gigabytes(torch):
    """Byte offsets past 32 bits: the last pages of a cache of 5.4 GB."""
    D, G, H, page = 128, 32, 2, 1024
    L = 1500
    n_pages = 5_400_000_000 // qcache.cache_bytes(1, H, D, page, G)
    c = qcache.QCache(n_pages, H, D, page_size=page, group=G)
    assert c.data.numel() > 1 << 32
    rng = np.random.default_rng(0)
    k, v = (rng.standard_normal((L, H, D)).astype(np.float16) for _ in range(2))
    b = Batch(torch, [L], [L], page)
    b.total, b.table = n_pages, np.array([[n_pages - 1, n_pages - 2]], np.int32)
    b.d_pages = torch.from_numpy(b.table).cuda()
    say("[gpu] cache past 4 GB")
    c.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), *b.args())
    got = c.read(*b.args(), n_tok=L, dtype=torch.float32)
    assert np.array_equal(got[0].cpu().numpy(), oc.held(k, G).astype(np.float32))
    b.new, b.start, b.n_tok = [1], np.array([0, 1]), 1
    q = queries(1, 4, D, seed=2)
    out = c.attend(torch.from_numpy(q).cuda(), b.d_lens, b.d_pages)
    check_attend(b, [(oc.quantise(k, G), oc.quantise(v, G))], q, out, 1 / math.sqrt(D), "past 4 GB")


@pytest.mark.gpu
def test_steps_captured_in_a_graph(torch):
    """write + attend captured once, replayed as the sequences grow, with eager work between the replays."""
    D, G, H, per, page, S = 128, 32, 2, 4, 16, 3
    start = [30, 0, 127]
    b = Batch(torch, [n + 20 for n in start], [1] * S, page, seed=2, one_each=True)
    rng = np.random.default_rng(1)
    c, _ = fill(torch, b, H, D, G, seed=5)
    eager = qcache.QCache(b.total, H, D, page_size=page, group=G)
    eager.data.copy_(c.data)
    k, v = (torch.zeros((S, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((S, H * per, D), dtype=torch.float16, device="cuda")
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    say("[gpu] captured write + attend")
    lens += 1
    c.write(k, v, lens, b.d_pages)
    c.attend(q, lens, b.d_pages)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.write(k, v, lens, b.d_pages)
        out = c.attend(q, lens, b.d_pages)
    for step in range(8):
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape)).astype(np.float16)))
        g.replay()
        torch.cuda.synchronize()
        eager.write(k, v, lens, b.d_pages)
        assert torch.equal(out, eager.attend(q, lens, b.d_pages)), f"replay {step}"
        lens += 1


@pytest.mark.gpu
def test_two_streams_at_once(torch):
    """Calls that overlap: each has its own workspace, and tensors made on one stream are used on another."""
    b = Batch(torch, [5000, 3000], [1, 1], 64, seed=1, one_each=True)
    c, enc = fill(torch, b, 2, 128, 32, seed=2)
    qs = [torch.from_numpy(queries(2, 8, 128, seed=i)).cuda() for i in range(8)]
    want = [c.attend(q, *b.args()) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    say("[gpu] attend on two streams")
    for _ in range(5):
        got = [c.attend(q, *b.args(), stream=streams[i % 2]) for i, q in enumerate(qs)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 8, 16])
def test_decoder_block_step(torch, batch):
    """A block's step as it is used: stacked q/k/v product with a bias, cache write, attention, output product
    added to the residual stream, gated product, down product added to it; against the same in fp64 from each
    operator's own FP16 inputs (the steps' own tests hold the tolerances; here, the run of them)."""
    from oracle import gemv
    from test_epilogue import act64, weights
    Hq, H, D, G, page = 4, 2, 64, 32, 16
    E = Hq * D
    w = {n: weights(f, m, kk) for n, f, m, kk in [("qkv", "block7b_u3", (Hq + 2 * H) * D, E), ("o", "mlp7b_lut3", E, E),
                                                  ("down", "mlp70b_lut4", E, 320)]}
    gate, up = weights("mlp7b_bpdq3", 320, E), weights("mlp7b_bpdq3", 320, E)
    up["codes_packed"] = up["codes_packed"][::-1].copy()
    w["gu"] = qgemv.interleave_rows(gate, up)
    plans = {n: qgemv.QGemv(x) for n, x in w.items()}
    lens = [40 + 3 * i for i in range(batch)]
    b = Batch(torch, lens, [1] * batch, page, seed=batch, one_each=True)
    c, enc = fill(torch, b, H, D, G, seed=7)
    x = torch.from_numpy(np.random.default_rng(batch).standard_normal((batch, E)).astype(np.float16)).cuda()
    bias = torch.randn((Hq + 2 * H) * D, device="cuda").half()
    say(f"[gpu] decoder block step, batch {batch}")
    qkv = plans["qkv"].run_epilogue(x, bias=bias)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, H * D, H * D], dim=1))
    c.write(k, v, *b.args())
    a = c.attend(q, *b.args())
    h = plans["o"].run_epilogue(a.view(batch, E), residual=x)
    m = plans["gu"].run_epilogue(h, act="silu", gated=True)
    y = plans["down"].run_epilogue(m, residual=h)
    n = lambda t: t.float().cpu().numpy().astype(np.float64)

    def near(got, want, A):
        # the products' 1e-4 A + 1e-6, FP16 rounding and, gated, both factors' errors: a factor 4 covers them
        tol = 4 * (1e-4 * A + 1e-6) + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
        assert np.all(np.abs(n(got) - want) <= tol + 2.0 ** -11 * tol)

    t, A = gemv.gemv(w["qkv"], n(x))
    near(qkv, t + n(bias), A)
    for s in range(batch):
        for i, new in enumerate((k, v)):
            e = oc.quantise(new[s].cpu().numpy(), G)
            for key in e:
                enc[s][i][key][lens[s] - 1] = e[key]
    check_attend(b, enc, q.cpu().numpy(), a, 1 / math.sqrt(D), "block")
    t, A = gemv.gemv(w["o"], n(a).reshape(batch, E))
    near(h, t + n(x), A)
    t, A = gemv.gemv(w["gu"], n(h))
    s = act64(t[:, 0::2], "silu")
    near(m, s * t[:, 1::2], A[:, 0::2] * np.abs(t[:, 1::2]) + np.abs(s) * A[:, 1::2] + 1e-4 * A[:, 0::2] * A[:, 1::2])
    t, A = gemv.gemv(w["down"], n(m))
    near(y, t + n(h), A)
    for p in plans.values():
        p.close()
