"""The norms around a block (qnorm_run) against the fp64 oracle.

Tolerance: oracle.block's for fp32 arithmetic, plus the rounding to the output's type: 2^-11 of the value in FP16 (2^-25
where it is subnormal), 2^-24 in fp32.  MX blocks must be those of the same call's fp32 output.
"""

import ctypes
import re

import numpy as np
import pytest

from dense_sparse_bit_amd import qgemv, qmx, qnorm
from gpu_checks import say
from oracle import block


# ---------------------------------------------------------------------------
# CPU
# ---------------------------------------------------------------------------
def test_library_exports_every_declared_symbol():
    with open(qgemv.HEADER.replace("qgemv.h", "qnorm.h")) as f:
        names = set(re.findall(r"^int (qnorm_\w+)\(", f.read(), re.M))
    assert names == {"qnorm_run"} and hasattr(qnorm.lib(), "qnorm_run")


def test_oracle_by_hand():
    x = np.array([[3.0, -4.0, 0.0, 0.0]])
    (h, _), (out, _) = block.norm(x, np.array([[1.0, 1.0, 1.0, 1.0]]), scale=2.0, pre=np.full(4, 2.0), eps=0.0)
    assert np.array_equal(h, [[5, -2, 2, 2]]) and np.allclose(out, 2 * h / np.sqrt(37 / 4))
    (h, _), (out, _) = block.norm(x, post=np.ones(4), gate=np.array([0.0, 1, 1, 1]), pre=np.ones(4), pre_bias=np.full(4, 7.0),
                                  kind="layer", eps=0.0)
    assert np.allclose(h, [[0, -3.75 / np.sqrt(99 / 16), 0.25 / np.sqrt(99 / 16), 0.25 / np.sqrt(99 / 16)]])
    assert np.isclose(out.mean(), 7) and np.isclose(out.var(), 1)


def args(**kw):
    r = lambda t=0, ld=64: qnorm.Rows(4096, t, ld)  # noqa: E731
    a = qnorm.Args(3, 64, 0, 1e-6, 1.0)
    a.y, a.h, a.pre, a.h_out, a.out = r(), r(), r(), r(), r()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


R = qnorm.Rows


@pytest.mark.parametrize("want,kw", [
    (-1, dict(rows=-1)), (-1, dict(cols=0)), (-3, dict(cols=60)), (-3, dict(cols=32776)), (-3, dict(rows=(1 << 26) + 1)),
    (-3, dict(kind=2)), (-1, dict(eps=-1.0)), (-1, dict(eps=float("nan"))), (-1, dict(eps=float("inf"))),
    (-1, dict(scale=float("inf"))), (-1, dict(y=R(), h=R())), (-1, dict(y=R(), gate=R(4096, 0, 64))),
    (-1, dict(y=R(), post=R(4096, 0, 0))), (-1, dict(post_bias=R(4096, 0, 0))), (-1, dict(pre=R(), out=R(), pre_bias=R(4096, 0, 0))),
    (-1, dict(pre=R())), (-1, dict(out=R())), (-1, dict(pre=R(), out=R(), h_out=R())), (-3, dict(y=R(4096, 2, 64))),
    (-1, dict(h=R(4104, 0, 64))), (-1, dict(h=R(4096, 0, 68))), (-1, dict(h_out=R(4096, 0, 56))), (-1, dict(out=R(4096, 0, 0))),
    (-3, dict(out=R(4096, 3, 64))), (-3, dict(gate=R(4096, 5, 64))), (-1, dict(pre=R(4100, 1, 0))),
    (-1, dict(out=R(4096 + 128, 16, 0))), (-3, dict(cols=40, out=R(4096, 17, 0))), (0, dict(rows=0))])
def test_refused(want, kw):
    """Refused before a launch; the pointers are never followed."""
    assert qnorm.lib().qnorm_run(ctypes.byref(args(**kw)), None) == want


@pytest.mark.parametrize("want,kw", [
    (-3, dict(rows=1 << 26, cols=512)), (-3, dict(rows=1 << 23, cols=2056)), (-3, dict(rows=1 << 20, cols=32768)),  # past a launch
    (-1, dict(out=R(4096, 0, 64))), (-1, dict(h_out=R(1 << 20, 1, 64))), (-1, dict(h_out=R(1 << 20, 0, 72))),
    (-1, dict(out=R(1 << 21, 1, 64))), (-1, dict(out=R(1 << 21, 16, 0))), (-1, dict(y=R(), out=R(4096, 0, 64)))])
def test_outputs_in_the_wrong_place_and_too_many_rows(want, kw):
    """y at 1 MiB, h at 2 MiB, h_out at 4096, out at 8192 unless given."""
    a = args(**{**dict(y=R(1 << 20, 0, 64), h=R(1 << 21, 0, 64), out=R(8192, 0, 64)), **kw})
    for r in (a.y, a.h, a.h_out, a.out):
        r.ld = r.ld if a.cols == 64 else a.cols
    assert qnorm.lib().qnorm_run(ctypes.byref(a), None) == want


def test_null():
    assert qnorm.lib().qnorm_run(None, None) == -1


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


def check(got, want, tol, what):
    f32 = "float32" in str(got.dtype)
    got = got.cpu().numpy().astype(np.float64)
    tol = tol + (2.0 ** -24 * np.abs(want) if f32 else np.maximum(2.0 ** -11 * np.abs(want), 2.0 ** -25)) * (1 + 2.0 ** -8)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = (np.abs(got - want) / (tol + 1e-300)).max()
    assert worst <= 1, f"{what}: worst |d| / tol = {worst:.3f}"


def data(torch, T, N, seed, f32=(False, False, False)):
    """Numpy arrays as the call takes them, and the same on the GPU."""
    rng = np.random.default_rng(seed)
    ty = [np.float32 if f else np.float16 for f in f32]
    a = {"y": (rng.standard_normal((T, N)) * np.exp(0.5 * rng.standard_normal(N))).astype(ty[0]),
         "h": (3 * rng.standard_normal((T, N)) + 0.5).astype(ty[1])}
    for k in ("post", "post_bias", "pre", "pre_bias"):
        a[k] = (1 + 0.3 * rng.standard_normal(N)).astype(ty[2])
    a["gate"] = rng.standard_normal((T, N)).astype(ty[2])
    a["gate1"] = rng.standard_normal(N).astype(ty[2])
    return a, {k: torch.from_numpy(v).cuda() for k, v in a.items()}


SIZES = [(1, 8), (3, 32), (5, 40), (17, 512), (4, 520), (9, 1024), (2, 1536), (33, 2048), (3, 2080), (1, 4096), (7, 5120),
         (2, 8192), (2, 8200), (1, 16384), (2, 28672), (1, 32768)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,N", SIZES)
def test_both_norms(torch, T, N, kind):
    say(f"[gpu] norm {T}x{N} {kind}")
    for f32, out_type in [((False, False, False), "fp16"), ((False, True, True), "fp32"), ((True, False, False), "fp32")]:
        a, g = data(torch, T, N, N + T, f32)
        kw = dict(post="post", post_bias="post_bias" if kind == "layer" else None, gate="gate", pre="pre", pre_bias="pre_bias")
        (h, dh), (o, do) = block.norm(a["y"], a["h"], **{k: v and a[v] for k, v in kw.items()}, scale=0.75, kind=kind, eps=1e-5)
        got_h, got = qnorm.norm(g["y"], g["h"], **{k: v and g[v] for k, v in kw.items()}, scale=0.75, kind=kind, eps=1e-5,
                                out_type=out_type)
        assert got_h.dtype == g["h"].dtype
        check(got_h, h, dh, "h")
        check(got, o, do, "out")


@pytest.mark.gpu
@pytest.mark.parametrize("what", [
    dict(y=0, pre=1), dict(h=0, pre=1), dict(pre=0), dict(pre=0, post=1), dict(pre=0, h=0, post=1), dict(h=0, gate1=1, pre=1),
    dict(gate1=1, pre=1), dict(post=1, gate=1, pre=1, pre_bias=1), dict(pre=1, scale=0.0), dict(y=0, pre=0, scale=-2.0)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,N", [(1, 4096), (6, 264), (3, 9000)])
def test_parts(torch, T, N, kind, what):
    """Every part may be missing."""
    a, g = data(torch, T, N, 3)
    kw = {"y": 1, "h": 1, **what}
    scale = kw.pop("scale", 1.0)
    names = {"gate1": "gate"}
    pick = lambda d: {names.get(k, k): d[k] for k, v in kw.items() if v}  # noqa: E731
    cpu, gpu = pick(a), pick(g)
    for d in (cpu, gpu):
        d.setdefault("y", None)
    (h, dh), o = block.norm(**cpu, scale=scale, kind=kind)
    got_h, got = qnorm.norm(**gpu, scale=scale, kind=kind)
    check(got_h, h, dh, "h")
    assert (got is None) == (o is None)
    if o is not None:
        check(got, *o, "out")
        none, again = qnorm.norm(**gpu, scale=scale, kind=kind, keep_h=False)
        assert none is None and torch.equal(again, got)


# rows enough for the tiles of 16 to be dealt out to the XCDs
MANY = [(512, 96), (525, 512), (641, 992), (1030, 4096), (700, 8192)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,N", [(1, 32), (5, 160), (17, 2080), (33, 4096), (3, 8224), (2, 32768)] + MANY)
def test_blocks(torch, T, N, kind, fmt):
    """out in MX blocks is what quantising the fp32 out gives, whatever the memory held, and the product takes it.  The blocks
    are rounded once, from more bits, so they may differ where the fp32 value is the middle between two elements or a block's largest
    is the largest element itself."""
    _, g = data(torch, T, N, N)
    kw = dict(y=g["y"], h=g["h"], post=g["post"], gate=g["gate"], pre=g["pre"], kind=kind)
    _, out = qnorm.norm(**kw, out_type="fp32")
    m = qmx.MxRows(T, N, fmt)
    m.data.fill_(255)
    _, got = qnorm.norm(**kw, out=m)
    assert got is m
    want = qmx.quantize(out, fmt)
    (gc, ge), (wc, we) = got.unpack(), want.unpack()
    largest, bits = (6.0, 1) if fmt == "e2m1" else (448.0, 3)
    u = out.double().view(T, -1, 32) / torch.exp2(we.double() - 127)[..., None]
    top = u.abs().amax(2)
    assert ((ge == we) | (top == largest)).all()
    same = (got.values() == want.values()).view(T, -1, 32) | (ge != we)[..., None]
    # an element's step at u, and whether u is in the middle of one
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=1.0 if fmt == "e2m1" else 2.0 ** -6))) - bits)
    assert (same | (torch.frac(u.abs() / step) == 0.5)).all()
    assert (~same).sum() + (ge != we).sum() <= 4 + 2e-6 * T * N
    want = got if not torch.equal(gc, wc) or not torch.equal(ge, we) else want
    w = qmx.QMx(qmx.quantize(torch.randn((24, N), device="cuda")))
    assert torch.equal(w.run(got), w.run(want))
    assert torch.isfinite(w.run(got)).all()


@pytest.mark.gpu
def test_strides_and_in_place(torch):
    T, N = 11, 1000
    _, g = data(torch, T, N, 8)
    kw = dict(post=g["post"], gate=g["gate1"], pre=g["pre"])
    h, out = qnorm.norm(g["y"], g["h"], **kw)
    wide = torch.full((T, 2 * N + 24), 7.0, device="cuda").half()
    y, hs = wide[:, 8:8 + N], wide[:, N + 16:2 * N + 16]
    y.copy_(g["y"])
    hs.copy_(g["h"])
    got = qnorm.norm(y, hs, **kw, h_out=hs, out=y)
    assert got[0] is hs and got[1] is y and torch.equal(hs, h) and torch.equal(y, out)
    edge = torch.ones_like(wide, dtype=torch.bool)
    edge[:, 8:8 + N] = edge[:, N + 16:2 * N + 16] = False
    assert (wide[edge] == 7).all()
    # one row broadcast
    row = g["y"][:1].expand(T, N)
    a, b = qnorm.norm(row.contiguous(), g["h"], **kw), None
    b = qnorm.norm(row, g["h"], **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_not_finite_and_zero_rows(torch):
    """A row with a NaN or an infinity is its own business; a row of zeros is 0 (the bias); eps keeps it finite."""
    y = torch.randn((6, 640), device="cuda").half()
    y[1, 5], y[3, 600] = float("nan"), float("inf")
    y[4] = 0
    pre, bias = torch.ones(640, device="cuda"), torch.full((640,), 0.5, device="cuda")
    for kind in ("rms", "layer"):
        _, out = qnorm.norm(y, pre=pre, pre_bias=bias, kind=kind)
        assert torch.isfinite(out[[0, 2, 4, 5]]).all() and (out[4] == 0.5).all()
        assert torch.isnan(out[1]).all() and torch.isnan(out[3]).any()
    assert qnorm.norm(y[:0], pre=pre)[1].shape == (0, 640)


@pytest.mark.gpu
def test_streams_and_capture(torch):
    for T, N in [(1, 8192), (40, 4096), (300, 256)]:
        _, g = data(torch, T, N, 1)
        kw = dict(post=g["post"], gate=g["gate"], pre=g["pre"])
        want = qnorm.norm(g["y"], g["h"], **kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = qnorm.norm(g["y"], g["h"], **kw, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        ho, o = (torch.empty_like(t) for t in want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qnorm.norm(g["y"], g["h"], **kw, h_out=ho, out=o)
        for _ in range(4):
            g["y"].normal_()
            ho.zero_()
            want = qnorm.norm(g["y"], g["h"], **kw)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(ho, want[0]) and torch.equal(o, want[1])


@pytest.mark.gpu
def test_python_refusals(torch):
    _, g = data(torch, 3, 64, 1)
    y, h = g["y"], g["h"]
    for bad in (lambda: qnorm.norm(None), lambda: qnorm.norm(y.double()), lambda: qnorm.norm(y, h[:2]), lambda: qnorm.norm(y.t()),
                lambda: qnorm.norm(y, h.cpu()), lambda: qnorm.norm(y, kind="batch"), lambda: qnorm.norm(y, eps=-1.0),
                lambda: qnorm.norm(y, scale=float("nan")), lambda: qnorm.norm(None, h, gate=g["gate"]),
                lambda: qnorm.norm(y, post_bias=g["post"]), lambda: qnorm.norm(y, pre=g["pre"][:32]),
                lambda: qnorm.norm(y, out=h), lambda: qnorm.norm(y, keep_h=False), lambda: qnorm.norm(y, pre=g["pre"], out_type="bf16"),
                lambda: qnorm.norm(y, pre=g["pre"], out=qmx.MxRows(3, 32)), lambda: qnorm.norm(y, gate=g["gate"][:, :32])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qgemv.QgemvError):
        qnorm.norm(y[:, :60].contiguous(), pre=g["pre"][:60].contiguous())
    with pytest.raises(qgemv.QgemvError):
        qnorm.norm(y[:, :40].contiguous(), pre=g["pre"][:40].contiguous(), out_type="fp16", h_out=y[:, 1:41])
