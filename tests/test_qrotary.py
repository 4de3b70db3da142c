"""Queries and keys turned by position, and appended to the 4-bit cache (qrotary_write), against the fp64 oracle.

A turned value is formed in 64 bits and rounded to fp32, then to FP16: it is off by 2^-11 (1 + 2^-13) of itself (2^-25 where
that is subnormal) and 2^-24 of its pair's length at most (the angle's own rounding is the definition's).  What the cache
holds must be, to the bit, what it holds for the same turned keys in FP16.
"""

import re

import numpy as np
import pytest

from dense_sparse_bit_amd import qcache, qgemv, qrotary
from gpu_checks import say
from oracle import block
from oracle import cache as oc


# ---------------------------------------------------------------------------
# CPU
# ---------------------------------------------------------------------------
def test_library_exports_every_declared_symbol():
    with open(qgemv.HEADER.replace("qgemv.h", "qrotary.h")) as f:
        names = set(re.findall(r"^int (qrotary_\w+)\(", f.read(), re.M))
    assert names == {"qrotary_write"} and hasattr(qrotary.lib(), "qrotary_write")


def test_oracle_turn_by_hand():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    f = [np.pi / 2, np.pi]
    assert np.allclose(block.turned(x, [[1]], f, "neighbours"), [[[-2, 1, -3, -4, 5, 6]]])
    assert np.allclose(block.turned(x, [[1]], f, "halves"), [[[-3, -2, 1, -4, 5, 6]]])
    assert np.allclose(block.turned(x, [[0], [1]], f, "halves", [0, 1]), [[[1, -2, 3, -4, 5, 6]]])
    assert np.array_equal(block.turned(x, [[3]], f, "halves", [1, -1]), x)


def test_calls_refused_on_the_host():
    """Everything that is refused before a launch; the pointers are never followed."""
    L, sh = qrotary.lib(), qcache.Shape(4, 2, 128, 64, 32)
    rows = qcache.Rows(4096, 0, 256, 128)
    ok = dict(rot_dim=128, style=0, axes=1, freqs=4096, pair_axis=None, positions=None)

    def call(sh=sh, cache=4096, heads=2, q=rows, out=rows, k=rows, v=rows, n_tok=2, n_seq=2, ro=True, **kw):
        r = qrotary._Rotary(*{**ok, **kw}.values())
        return L.qrotary_write(sh, cache, qcache.Seqs(n_seq, n_tok, 1, None, 4096, 4096), r if ro else None, heads, q, out, k, v, None)

    assert call(ro=False) == -1 and call(cache=None) == -1 and call(sh=qcache.Shape(4, 2, 96, 64, 32)) == -3
    assert call(rot_dim=0) == -3 and call(rot_dim=24) == -3 and call(rot_dim=144) == -3 and call(rot_dim=-16) == -3
    assert call(style=2) == -3 and call(style=-1) == -3 and call(axes=0) == -3 and call(axes=17, positions=4096) == -3
    assert call(freqs=None) == -1 and call(freqs=4100) == -1 and call(pair_axis=4098) == -1 and call(positions=4098) == -1
    assert call(axes=2) == -1  # no positions
    assert call(heads=-1) == -1 and call(heads=65536) == -3
    for bad, want in [(None, -1), (qcache.Rows(None, 0, 256, 128), -1), (qcache.Rows(4104, 0, 256, 128), -1),
                      (qcache.Rows(4096, 2, 256, 128), -3), (qcache.Rows(4096, 0, 252, 128), -1)]:
        assert call(q=bad) == want and call(out=bad) == want and call(k=bad) == want and call(v=bad) == want
    assert call(out=qcache.Rows(4096, 0, 0, 128)) == -1 and call(out=qcache.Rows(4096, 0, 256, 64)) == -1
    assert call(v=qcache.Rows(4096, 1, 256, 128)) == -1 and call(n_tok=3) == -1
    assert call(n_seq=0, n_tok=0) == 0 and call(n_seq=0, n_tok=0, rot_dim=8) == -3
    assert call(sh=qcache.Shape(4, 65535, 128, 64, 32), n_seq=1 << 20, n_tok=1 << 20) == -3  # past a launch


def test_overlapping_queries_are_refused():
    """q_out's vectors may lie token by token or head by head, with gaps, and not in each other."""
    L, sh, ok = qrotary.lib(), qcache.Shape(4, 2, 128, 64, 32), qcache.Rows(4096, 0, 256, 128)
    r = qrotary._Rotary(8, 0, 1, 4096, None, None)  # refused for rot_dim once all else is in order: -3 comes before q_out
    assert L.qrotary_write(sh, 4096, qcache.Seqs(5, 5, 1, None, 4096, 4096), r, 3, ok, ok, ok, ok, None) == -3
    r.rot_dim = 128
    for ts, hs in [(128, 128), (256, 128), (128, 512), (376, 128), (128, 632), (-512, 128), (512, -128), (8, 1024), (1024, 8),
                   (0, 128), (640, 0)]:
        bad = qcache.Rows(4096, 0, ts, hs)
        assert L.qrotary_write(sh, 4096, qcache.Seqs(5, 5, 1, None, 4096, 4096), r, 3, ok, bad, ok, ok, None) == -1, (ts, hs)


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


def table(torch, lens, page, seed=0, spare=2):
    need = [-(-max(n, 0) // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    out = np.full((len(lens), max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        out[s, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(out).cuda(), sum(need) + spare


def i32(torch, a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def freqs(rot, base=10000.0):
    return base ** (-np.arange(rot // 2) / (rot // 2))


def check_turned(got, x, positions, f, style, pair_axis=None):
    want = block.turned(x, positions, f, style, pair_axis)
    got = got.cpu().numpy().astype(np.float64)
    f16 = np.maximum(2.0 ** -11 * (1 + 2.0 ** -12) * np.abs(want), 2.0 ** -25 * (1 + 2.0 ** -12))
    length = np.abs(np.asarray(x, dtype=np.float64)).max() * 2 ** 0.5
    assert (np.abs(got - want) <= f16 + 2.0 ** -50 * length).all(), np.abs(got - want).max()


SHAPES = [  # D, group, rot, style, heads, per, page
    (128, 32, 128, "halves", 2, 4, 64), (128, 64, 64, "halves", 3, 1, 16), (128, 128, 32, "neighbours", 1, 5, 32),
    (64, 32, 64, "neighbours", 4, 2, 16), (64, 64, 16, "halves", 2, 3, 64), (64, 32, 48, "halves", 1, 8, 128),
    (256, 64, 256, "halves", 2, 2, 32), (256, 128, 64, "neighbours", 1, 3, 16), (256, 32, 80, "halves", 2, 1, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lens,new", [([5], [5]), ([40, 16, 1, 0, 33], [40, 3, 1, 0, 17]), ([100, 7, 1000], [1, 1, 1]),
                                      ([129], [65])])
@pytest.mark.parametrize("D,G,rot,style,H,per,page", SHAPES)
def test_write(torch, D, G, rot, style, H, per, page, lens, new, f32):
    rng = np.random.default_rng(D + rot + len(lens))
    T, f = sum(new), freqs(rot)
    ty = np.float32 if f32 else np.float16
    k, v = ((rng.standard_normal((T, H, D)) + 2 * rng.standard_normal((H, D))).astype(ty) for _ in range(2))
    q = rng.standard_normal((T, H * per, D)).astype(ty)
    pages, total = table(torch, lens, page)
    start = None if all(n == 1 for n in new) else i32(torch, np.concatenate([[0], np.cumsum(new)]))
    own = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])[None]
    rot_ = qrotary.Rotary(f, style)
    c, plain = (qcache.QCache(total, H, D, page_size=page, group=G) for _ in range(2))
    c.data.zero_()
    plain.data.zero_()
    say(f"[gpu] rotary D {D} rot {rot} {style} lens {lens} new {new} {ty.__name__}")
    gk, gv, gq = (torch.from_numpy(a).cuda() for a in (k, v, q))
    out = rot_.write(c, gq, gk, gv, i32(torch, lens), pages, start)
    assert out.dtype == torch.float16
    check_turned(out, q, own, f, style)
    # keys: turned as queries are, then what the cache holds of them in FP16
    other = qcache.QCache(total, H, D, page_size=page, group=G)
    tk = rot_.write(other, gk, gk, gv, i32(torch, lens), pages, start)
    check_turned(tk, k, own, f, style)
    plain.write(tk, gv.half(), i32(torch, lens), pages, start)
    assert torch.equal(c.data, plain.data)
    got = c.read(i32(torch, lens), pages, start, n_tok=T, dtype=torch.float32)
    assert np.array_equal(got[0].cpu().numpy(), oc.held(tk.cpu().numpy(), G).astype(np.float32))
    # in place, and fp32 out
    at = rot_.write(other, gq, gk, gv, i32(torch, lens), pages, start, out=torch.empty_like(gq, dtype=torch.float32))
    assert torch.equal(at.half(), out)
    inplace = gq.clone()
    assert rot_.write(other, inplace, gk, gv, i32(torch, lens), pages, start, out=inplace) is inplace
    assert torch.equal(inplace.half(), out)
    # keys and values only
    other.data.zero_()
    assert rot_.write(other, None, gk, gv, i32(torch, lens), pages, start) is None
    assert torch.equal(other.data, c.data)


@pytest.mark.gpu
@pytest.mark.parametrize("style", ["halves", "neighbours"])
@pytest.mark.parametrize("axes", [1, 2, 3])
def test_axes(torch, axes, style):
    """Positions of several axes, also negative and far ones; a pair of an axis that is none stays."""
    rng = np.random.default_rng(axes)
    D, H, T, lens = 128, 2, 50, [20, 64]
    f = freqs(D)
    ax = rng.integers(0, axes + 1, D // 2) if axes > 1 else None
    if ax is not None:
        ax[3] = -1
    pos = rng.integers(-1000, 2 ** 20, (axes, T)).astype(np.int32)
    pos[0, 0] = 2 ** 31 - 1
    q, k, v = (rng.standard_normal((T, n, D)).astype(np.float16) for n in (6, H, H))
    pages, total = table(torch, lens, 16)
    c = qcache.QCache(total, H, D, page_size=16)
    start = i32(torch, [0, 20, 50])
    r = qrotary.Rotary(f, style, ax)
    args = [torch.from_numpy(a).cuda() for a in (q, k, v)] + [i32(torch, lens), pages, start]
    out = r.write(c, *args, positions=i32(torch, pos))
    check_turned(out, q, pos, f, style, ax)
    tk = r.write(c, args[1], args[1], *args[2:], positions=i32(torch, pos))
    got = c.read(*args[3:], n_tok=T, dtype=torch.float32)
    assert np.array_equal(got[0].cpu().numpy(), oc.held(tk.cpu().numpy(), 32).astype(np.float32))
    assert np.array_equal(got[1].cpu().numpy(), oc.held(v, 32).astype(np.float32))
    if axes == 1:
        assert torch.equal(out, r.write(c, *args, positions=i32(torch, pos[0])))


@pytest.mark.gpu
def test_padding_pages_and_strides(torch):
    """Rows of padding stay, rows without a page are turned but not stored, views of a stacked product are taken as they are."""
    rng = np.random.default_rng(7)
    D, H, Hq, page = 64, 2, 4, 16
    lens, new = [30, 5, 18, 3], [30, 5, 2, 6]  # the last one has rows before its first position
    T, pad = sum(new), 3
    f = freqs(D)
    qkv = torch.from_numpy(rng.standard_normal((T + pad, (Hq + 2 * H) * D)).astype(np.float16)).cuda()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, H * D, H * D], dim=1))
    pages = i32(torch, [[0, -1], [99, 99], [2, 1], [3, -1]])
    c = qcache.QCache(4, H, D, page_size=page)
    c.data.fill_(0x5A)
    before = c.data.clone()
    start = i32(torch, np.concatenate([[0], np.cumsum(new)]))
    out = torch.full((T + pad, Hq + 1, D), 7.0, device="cuda").half()
    r = qrotary.Rotary(f)
    r.write(c, q, k, v, i32(torch, lens), pages, start, out=out[:, :Hq])
    own = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])[None]
    check_turned(out[:T, :Hq], q[:T].cpu().numpy(), own, f, "halves")
    assert (out[T:] == 7).all() and (out[:, Hq] == 7).all()
    tk = r.write(qcache.QCache(4, H, D, page_size=page), k.contiguous(), k, v, i32(torch, lens), pages, start)
    want = qcache.QCache(4, H, D, page_size=page)
    want.data.copy_(before)
    want.write(tk, v, i32(torch, lens), pages, start)
    assert torch.equal(c.data, want.data)
    # in place in the stacked product
    again = r.write(c, q, k, v, i32(torch, lens), pages, start, out=q)
    assert torch.equal(again[:T], out[:T, :Hq])


@pytest.mark.gpu
def test_not_finite(torch):
    """An infinity makes its pair NaN or infinite, and its key's group NaN in the cache; other rows are not touched."""
    rng = np.random.default_rng(2)
    k, v = (rng.standard_normal((20, 1, 64)).astype(np.float16) for _ in range(2))
    k[4, 0, 3] = np.inf
    pages, total = table(torch, [20], 16)
    c = qcache.QCache(total, 1, 64, page_size=16)
    gk = torch.from_numpy(k).cuda()
    args = (gk, torch.from_numpy(v).cuda(), i32(torch, [20]), pages, i32(torch, [0, 20]))
    out = qrotary.Rotary(freqs(64)).write(c, gk, *args)
    bad = ~torch.isfinite(out).cpu().numpy()
    assert bad[4, 0, [3, 35]].all() and bad.sum() == 2
    held = c.read(*args[2:], n_tok=20)[0].cpu().numpy()
    assert np.isnan(held[4]).all() and np.isfinite(np.delete(held, 4, axis=0)).all()


@pytest.mark.gpu
def test_streams_and_capture(torch):
    """A captured call follows lens, pages, positions and rows over several replays."""
    rng = np.random.default_rng(9)
    D, H, S = 128, 2, 3
    r = qrotary.Rotary(freqs(D))
    for start in (None, [0, 2, 9, 20]):
        T = S if start is None else 20
        q, k, v = (torch.randn((T, n, D), device="cuda").half() for n in (4, H, H))
        lens, pages = i32(torch, [40, 30, 50]), torch.arange(12, dtype=torch.int32, device="cuda").view(S, 4)
        st = None if start is None else i32(torch, start)
        c, d = (qcache.QCache(12, H, D, page_size=16) for _ in range(2))
        c.data.zero_()
        d.data.zero_()
        want = r.write(d, q, k, v, lens, pages, st)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = r.write(c, q, k, v, lens, pages, st, stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(c.data, d.data)
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.write(c, q, k, v, lens, pages, st, out=out)
        for i in range(4):
            q.normal_()
            k.normal_()
            lens += 3
            want = r.write(d, q, k, v, lens, pages, st)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(c.data, d.data)


@pytest.mark.gpu
def test_python_refusals(torch):
    c = qcache.QCache(2, 2, 64, page_size=16)
    r = qrotary.Rotary(freqs(64))
    q, k = torch.randn((3, 4, 64), device="cuda").half(), torch.randn((3, 2, 64), device="cuda").half()
    lens, pages = i32(torch, [1, 2, 3]), i32(torch, [[0], [1], [-1]])
    pos = i32(torch, [1, 2, 3])
    for bad in (lambda: qrotary.Rotary(freqs(64), "thirds"), lambda: qrotary.Rotary(freqs(64), pair_axis=[0]),
                lambda: qrotary.Rotary([freqs(64)]), lambda: qrotary.Rotary(freqs(64), device="cpu").write(c, q, k, k, lens, pages),
                lambda: r.write(c, q[:2], k, k, lens, pages), lambda: r.write(c, q, k[:, :1], k, lens, pages),
                lambda: r.write(c, q, k, k.float(), lens, pages), lambda: r.write(c, q, k, k, lens, pages, positions=pos[:2]),
                lambda: r.write(c, q, k, k, lens, pages, positions=pos.long()), lambda: r.write(c, None, k, k, lens, pages, out=q),
                lambda: r.write(c, q, k, k, lens, pages, out=q[:, :2]), lambda: r.write(c, q.double(), k, k, lens, pages),
                lambda: r.write(c, q.expand(3, 4, 64)[:, :1].expand(3, 4, 64), k, k, lens, pages, out=q[:, :1].expand(3, 4, 64))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qgemv.QgemvError):
        qrotary.Rotary(freqs(128)).write(c, q, k, k, lens, pages)
