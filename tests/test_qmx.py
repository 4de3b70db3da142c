"""Rows in MX blocks (qmx_quantize, qmx_values, qmx_pack, qmx_unpack) and their product (qmx_run) against the fp64 oracle.

Blocks are defined to the bit: codes and exponent bytes must be equal.  The
product's tolerance is oracle.mx.product's, plus the rounding to the output's
type: 2^-11 of the value in FP16 (2^-25 where it is subnormal), 2^-24 in fp32.
"""

import ctypes
import re

import numpy as np
import pytest

from dense_sparse_bit_amd import qgemv, qmx
from gpu_checks import say
from oracle import mx

FORMATS = ["e2m1", "e4m3"]


# ---------------------------------------------------------------------------
# CPU
# ---------------------------------------------------------------------------
def test_library_exports_every_declared_symbol():
    with open(qgemv.HEADER.replace("qgemv.h", "qmx.h")) as f:
        names = set(re.findall(r"^int (qmx_\w+)\(", f.read(), re.M))
    assert names == {"qmx_bytes", "qmx_quantize", "qmx_values", "qmx_pack", "qmx_unpack", "qmx_run_ws", "qmx_run"}
    for n in names:
        assert hasattr(qmx.lib(), n), n


def test_oracle_grid_and_rounding():
    assert list(mx.grid("e2m1")) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    g = mx.grid("e4m3")
    assert len(g) == 127 and g[1] == 2.0 ** -9 and g[8] == 2.0 ** -6 and g[-1] == 448 and np.all(np.diff(g) > 0)
    x = np.zeros((1, 32))
    x[0, :12] = [6, 5, 4.999, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -0.2500001, -5]  # ties to the even code
    codes, exps = mx.quantise(x, "e2m1")
    assert exps[0, 0] == 127
    assert list(mx.values(codes, exps, "e2m1")[0, :12]) == [6, 4, 4, 4, 2, 2, 1, 1, 0, 0, -0.5, -4]
    for top, no_clip, clip in [(6, 127, 127), (6.001, 128, 127), (7.99, 128, 127), (4, 127, 127), (3.99, 127, 126),
                               (3, 126, 126), (3.01, 127, 126)]:
        x[0] = 0
        x[0, 5] = -top
        assert mx.quantise(x, "e2m1")[1][0, 0] == no_clip and mx.quantise(x, "e2m1", True)[1][0, 0] == clip, top
    x[0, 5] = 7.9
    assert mx.values(*mx.quantise(x, "e2m1", True), "e2m1")[0, 5] == 6
    x[0, 5] = np.nan
    assert np.isnan(mx.values(*mx.quantise(x, "e2m1"), "e2m1")).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_oracle_nearest(fmt):
    """Without clipping every value is within half a step of the grid around it."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 64)) * 10.0 ** rng.integers(-8, 8, (40, 1))
    codes, exps = mx.quantise(x, fmt)
    v = mx.values(codes, exps, fmt)
    step = np.repeat(2.0 ** (exps.astype(float) - 127), 32, axis=1)
    half = np.maximum(np.abs(x) * (2.0 ** -2 if fmt == "e2m1" else 2.0 ** -4), step * (0.25 if fmt == "e2m1" else 2.0 ** -10))
    assert np.all(np.abs(v - x) <= half)
    assert np.all(np.abs(v) <= mx.grid(fmt)[-1] * step)


@pytest.mark.parametrize("rows,cols,fmt", [(1, 32, "e2m1"), (16, 128, "e2m1"), (17, 160, "e4m3"), (4096, 11008, "e2m1")])
def test_bytes(rows, cols, fmt):
    n = ctypes.c_size_t(0)
    assert qmx.lib().qmx_bytes(qmx.Shape(rows, cols, qmx.FORMAT[fmt]), n) == 0
    tiles, chunks = -(-rows // 16), -(-cols // 128)
    assert n.value == tiles * (chunks * (1024 if fmt == "e2m1" else 2048) + -(-chunks // 4) * 256)


@pytest.mark.parametrize("shape,want", [
    ((-1, 32, 0), -1), ((1, 0, 0), -1), ((1, -32, 0), -1), ((1, 48, 0), -3), ((1, 1 << 21, 0), -3),
    ((1 << 27, 32, 0), -3), ((1, 32, 2), -3), ((1, 32, -1), -3), ((1 << 26, 1 << 20, 0), -3)])
def test_shapes_refused(shape, want):
    n = ctypes.c_size_t(0)
    L = qmx.lib()
    assert L.qmx_bytes(qmx.Shape(*shape), n) == want
    assert L.qmx_quantize(qmx.Shape(*shape), 4096, 4096, 0, 64, 0, None) == want
    assert L.qmx_values(qmx.Shape(*shape), 4096, 4096, 0, 1 << 22, None) == want
    assert L.qmx_pack(qmx.Shape(*shape), 4096, 4096, 4096, None) == want


def test_calls_refused_on_the_host():
    """Everything that is refused before a launch; the pointers are never followed."""
    L, sh = qmx.lib(), qmx.Shape(3, 64, 0)
    assert L.qmx_bytes(sh, None) == -1 and L.qmx_bytes(None, ctypes.c_size_t(0)) == -1
    for f in (lambda *a: L.qmx_quantize(sh, *a, 0, None), lambda *a: L.qmx_values(sh, *a, None)):
        assert f(None, 4096, 0, 64) == -1 and f(4096 + 128, 4096, 0, 64) == -1
        assert f(4096, None, 0, 64) == -1 and f(4096, 4104, 0, 64) == -1 and f(4096, 4096, 0, 68) == -1
        assert f(4096, 4096, 2, 64) == -3
    assert L.qmx_values(sh, 4096, 4096, 0, 56, None) == -1  # rows overlap
    for f in (L.qmx_pack, L.qmx_unpack):
        assert f(sh, None, 4096, 4096, None) == -1 and f(sh, 4096, None, 4096, None) == -1
        assert f(sh, 4096, 4096, None, None) == -1 and f(sh, 4096, 4098, 4096, None) == -1

    def run(w=qmx.Shape(6, 64, 0), blocks=4096, data=4096, rows=3, fmt=0, x_type=-1, ldx=0, y=4096, ws=4096, n=1 << 20,
            epi=True, **kw):
        e = qgemv.Epilogue()
        for k, v in kw.items():
            setattr(e, k, v)
        return L.qmx_run(w, blocks, qmx.Input(data, rows, fmt, x_type, ldx), y, e if epi else None, ws, n, None)

    assert run(w=qmx.Shape(6, 64, 1)) == -3 and run(w=qmx.Shape(0, 64, 0)) == -1 and run(w=qmx.Shape(6, 60, 0)) == -3
    assert run(blocks=None) == -1 and run(blocks=4096 + 64) == -1 and run(data=None) == -1 and run(data=4096 + 64) == -1
    assert run(y=None) == -1 and run(y=4097) == -1 and run(y=4098, y_type=1) == -1 and run(epi=False) == -1
    assert run(rows=-1) == -1 and run(rows=1 << 27) == -3 and run(fmt=2) == -3 and run(x_type=2) == -3
    assert run(act=5) == -3 and run(act=-1) == -3 and run(y_type=2) == -3 and run(bias_type=3) == -3
    assert run(w=qmx.Shape(5, 64, 0), gated=1) == -3 and run(ldy=5) == -1 and run(residual=4096, ldr=5) == -1
    assert run(residual=4097) == -1 and run(bias=4097) == -1
    assert run(x_type=0, ldx=64, data=4104) == -1 and run(x_type=0, ldx=68) == -1
    few = dict(rows=17, x_type=0, ldx=64)
    assert run(**few, ws=None) == -1 and run(**few, ws=4096 + 32) == -1 and run(**few, n=64) == -5
    assert run(w=qmx.Shape(1 << 20, 64, 0), rows=1 << 17, ldy=1 << 20) == -3  # past a launch
    n = ctypes.c_size_t(0)
    x = qmx.Input(None, 17, 0, 0, 64)
    assert L.qmx_run_ws(qmx.Shape(6, 64, 0), x, qgemv.Epilogue(), n) == 0 and n.value > 0
    assert L.qmx_run_ws(qmx.Shape(6, 64, 0), qmx.Input(None, 17, 0, -1, 0), qgemv.Epilogue(), n) == 0 and n.value == 0
    assert L.qmx_run_ws(qmx.Shape(6, 64, 0), x, qgemv.Epilogue(), None) == -1
    assert L.qmx_run_ws(qmx.Shape(6, 64, 0), None, qgemv.Epilogue(), n) == -1
    assert run(rows=0, data=None, y=None, ws=None, n=0) == 0  # no rows: nothing is done
    assert L.qmx_quantize(qmx.Shape(0, 64, 0), None, None, 0, 64, 0, None) == 0


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


def plain(m):
    """Codes one a byte and exponent bytes of MxRows, as the oracle has them."""
    codes, exps = (a.cpu().numpy() for a in m.unpack())
    if m.fmt == "e2m1":
        codes = np.stack([codes & 15, codes >> 4], axis=2).reshape(m.rows, m.cols)
    return codes, exps


def poisoned(torch, rows, cols, fmt):
    """MxRows over memory that holds NaN blocks wherever nothing is written."""
    m = qmx.MxRows(rows, cols, fmt)
    m.data.fill_(255)
    return m


def hard_rows(rng, T, K):
    """Values of many sizes, with zeros, ties, and blocks at the ends of FP16."""
    x = rng.standard_normal((T, K)) * np.repeat(2.0 ** rng.integers(-20, 10, (T, K // 32)), 32, axis=1)
    x[rng.random((T, K)) < 0.1] = 0
    b = x.reshape(-1, 32)
    for i in range(0, len(b), 7):  # exact halves of a grid, so that ties occur
        b[i] = rng.integers(-24, 25, 32) * 2.0 ** rng.integers(-14, 3) / 4
    b[0] = 0
    b[len(b) // 2, 3] = -65504
    b[-1] = 2.0 ** -24 * rng.integers(-3, 4, 32)
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K", [(1, 32), (1, 4096), (3, 160), (16, 128), (17, 544), (33, 96), (100, 2080)])
@pytest.mark.parametrize("f32", [False, True])
def test_quantize(torch, T, K, fmt, clip, f32):
    rng = np.random.default_rng(T * 1000 + K + clip)
    x = hard_rows(rng, T, K).astype(np.float32 if f32 else np.float16)
    if f32:
        x[0, :4] = [3e38, -1e-38, 2.0 ** -130, 1.1754944e-38]
        x[-1, -32:] = 2.0 ** -127 * rng.integers(-9, 10, 32)  # below the smallest power of two
    codes, exps = mx.quantise(x, fmt, clip)
    say(f"[gpu] quantize {T}x{K} {fmt}")
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.float32 if f32 else torch.float16, device="cuda")
    wide[:, 8:8 + K] = torch.from_numpy(x).cuda()
    m = qmx.quantize(wide[:, 8:8 + K], fmt, clip, out=poisoned(torch, T, K, fmt))
    got, gexp = plain(m)
    assert np.array_equal(gexp, exps)
    # the sign of a zero element is not part of the value
    sign = 8 if fmt == "e2m1" else 128
    assert np.array_equal(np.where(got % sign, got, 0), np.where(codes % sign, codes, 0))
    v = mx.values(codes, exps, fmt)
    for dt in (torch.float32, torch.float16):
        with np.errstate(over="ignore"):
            want = v.astype(np.float32 if dt == torch.float32 else np.float16)
        assert np.array_equal(m.values(dt).cpu().numpy(), want)
    again = qmx.MxRows.pack(*m.unpack(), fmt)
    assert all(torch.equal(a, b) for a, b in zip(again.unpack(), m.unpack()))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_not_finite(torch, fmt):
    x = torch.randn((5, 128), device="cuda")
    x[1, 40], x[2, 0], x[4, 127] = float("nan"), float("inf"), -float("inf")
    v = qmx.quantize(x, fmt).values().cpu().numpy()
    bad = np.zeros((5, 4), dtype=bool)
    bad[1, 1] = bad[2, 0] = bad[4, 3] = True
    assert np.array_equal(np.isnan(v), np.repeat(bad, 32, axis=1))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_pack_every_code(torch, fmt):
    """All codes with all exponent bytes, through pack, values and unpack."""
    n = 16 if fmt == "e2m1" else 256
    codes = np.tile(np.arange(n, dtype=np.uint8), 256 * 32 // n).reshape(256 // 8, 8 * 32)
    exps = np.arange(256, dtype=np.uint8).reshape(32, 8)
    m = qmx.MxRows.pack(torch.from_numpy(mx.pack_bytes(codes, fmt)).cuda(), torch.from_numpy(exps).cuda(), fmt)
    got, gexp = plain(m)
    assert np.array_equal(got, codes) and np.array_equal(gexp, exps)
    with np.errstate(over="ignore"):
        want = mx.values(codes, exps, fmt).astype(np.float32)
    assert np.array_equal(m.values().cpu().numpy(), want, equal_nan=True)
    out = torch.full((32, 8 * 32 + 8), 7.0, device="cuda")
    m.values(out=out[:, :8 * 32])
    assert (out[:, 8 * 32:] == 7).all()


def weights(rng, M, K):
    codes = rng.integers(0, 16, (M, K)).astype(np.uint8)
    exps = rng.integers(118, 123, (M, K // 32)).astype(np.uint8)
    return codes, exps


def make(torch, rng, T, M, K, fmt, rows):
    """(plan, x as the call takes it, values of x, values of W)"""
    wc, we = weights(rng, M, K)
    plan = qmx.QMx(qmx.MxRows.pack(torch.from_numpy(mx.pack_bytes(wc, "e2m1")).cuda(), torch.from_numpy(we).cuda()))
    x = (rng.standard_normal((T, K)) * np.exp(0.5 * rng.standard_normal(K))).astype(np.float16)
    xv = mx.values(*mx.quantise(x, fmt), fmt)
    xt = torch.from_numpy(x).cuda()
    if not rows:
        xt = qmx.quantize(xt, fmt, out=poisoned(torch, T, K, fmt))
    return plan, xt, xv, mx.values(wc, we, "e2m1")


def check(got, want, tol, f32):
    got = got.cpu().numpy().astype(np.float64)
    tol = tol + (2.0 ** -24 * np.abs(want) if f32 else np.maximum(2.0 ** -11 * np.abs(want), 2.0 ** -25)) * (1 + 2.0 ** -8)
    assert got.shape == want.shape and np.isfinite(got).all()
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, f"worst |dy| / tol = {worst:.3f}"


SIZES = [(1, 16, 32), (1, 1, 64), (1, 4096, 4096), (2, 50, 160), (5, 300, 1024), (8, 130, 544), (16, 512, 2080), (17, 40, 512),
         (31, 256, 640), (33, 1000, 1184), (64, 384, 1536), (100, 272, 2176), (129, 513, 416), (257, 264, 1024), (300, 1100, 800)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("T,M,K", SIZES)
def test_product(torch, T, M, K, fmt, rows):
    rng = np.random.default_rng(T + M + K)
    say(f"[gpu] product T {T} M {M} K {K} {fmt} {'rows' if rows else 'blocks'}")
    plan, x, xv, wv = make(torch, rng, T, M, K, fmt, rows)
    want, tol = mx.product(xv, wv)
    y = plan.run(x, fmt, dtype=torch.float32)
    check(y, want, tol, True)
    assert torch.equal(y, plan.run(x, fmt, dtype=torch.float32))
    check(plan.run(x, fmt), want, tol, False)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,M,K", [(1, 48, 1024), (20, 64, 4096), (140, 144, 992)])
def test_product_of_wide_ranges(torch, T, M, K, fmt):
    """Every element of the formats, and powers of two 2^40 apart within a row: sums keep fp32's accuracy."""
    rng = np.random.default_rng(K)
    wc = rng.integers(0, 16, (M, K)).astype(np.uint8)
    we = rng.integers(107, 148, (M, K // 32)).astype(np.uint8)
    xc = rng.integers(0, 16 if fmt == "e2m1" else 256, (T, K)).astype(np.uint8)
    xc[xc % 128 == 127] -= 1
    xe = rng.integers(107, 148, (T, K // 32)).astype(np.uint8)
    gpu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    plan = qmx.QMx(qmx.MxRows.pack(gpu(mx.pack_bytes(wc, "e2m1")), gpu(we)))
    x = qmx.MxRows.pack(gpu(mx.pack_bytes(xc, fmt)), gpu(xe), fmt)
    want, tol = mx.product(mx.values(xc, xe, fmt), mx.values(wc, we, "e2m1"))
    check(plan.run(x, dtype=torch.float32), want, tol, True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,M,K", [(64, 24576, 1024), (300, 4096, 4096), (1000, 8192, 2048), (1030, 4096, 8192), (2050, 22016, 1184),
                                   (4000, 8192, 4096), (8192, 14336, 512)])
def test_product_of_many_workgroups(torch, T, M, K, fmt):
    """Every output of products that fill the card several times over, three times in a row: the copies through LDS have all
    landed when they are read."""
    rng = np.random.default_rng(T + K)
    say(f"[gpu] product T {T} M {M} K {K} {fmt}")
    wc, we = torch.randint(0, 256, (M, K // 2), device="cuda", dtype=torch.uint8), torch.randint(
        118, 123, (M, K // 32), device="cuda", dtype=torch.uint8)
    w = qmx.MxRows.pack(wc, we)
    plan, x = qmx.QMx(w), qmx.quantize(torch.randn((T, K), device="cuda") * float(rng.uniform(0.5, 2)), fmt)
    xv, wv = x.values().double(), w.values().double()
    want = xv @ wv.t()
    tol = ((128 + K / 128 + 16) * 2.0 ** -24 + 2.0 ** -24) * (xv.abs() @ wv.abs().t()) + 2.0 ** -126  # and the output's rounding
    ys = [plan.run(x, dtype=torch.float32) for _ in range(3)]
    for y in ys:
        worst = ((y.double() - want).abs() / tol).max().item()
        assert worst <= 1, f"worst |dy| / tol = {worst:.3f}"
        assert torch.equal(y, ys[0])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,M,K", [(1, 96, 256), (16, 130, 512), (19, 70, 352), (70, 522, 1024), (260, 514, 640)])
def test_epilogue(torch, T, M, K, gated, act):
    """Bias, activation, gate and strided residual and output; what lies between the rows stays."""
    rng = np.random.default_rng(M + T)
    f32 = (T + len(act)) % 2 == 0
    plan, x, xv, wv = make(torch, rng, T, M, K, "e4m3" if T % 2 else "e2m1", T != 19)
    fmt = "e4m3" if T % 2 else "e2m1"
    mo = M // 2 if gated else M
    bias = rng.standard_normal(M).astype(np.float32 if not f32 else np.float16)
    res = rng.standard_normal((T, mo)).astype(np.float16 if not f32 else np.float32)
    want, tol = mx.product(xv, wv, bias, act, gated, res)
    dt = torch.float32 if f32 else torch.float16
    out = torch.full((T + 2, mo + 5), 7.0, dtype=dt, device="cuda")
    wide = torch.full((T, mo + 3), float("nan"), dtype=torch.from_numpy(res).dtype, device="cuda")
    wide[:, 1:1 + mo] = torch.from_numpy(res).cuda()
    say(f"[gpu] epilogue T {T} M {M} K {K} {act} gated {gated}")
    y = out[1:1 + T, 2:2 + mo]
    plan.run(x, fmt, torch.from_numpy(bias).cuda(), act, gated, wide[:, 1:1 + mo], out=y)
    check(y, want, tol, f32)
    edge = torch.ones_like(out, dtype=torch.bool)
    edge[1:1 + T, 2:2 + mo] = False
    assert (out[edge] == 7).all()
    # dense, and the residual in place
    dense = torch.from_numpy(res).cuda().to(dt)
    want, tol = mx.product(xv, wv, bias, act, gated, dense.cpu().numpy())
    plan.run(x, fmt, torch.from_numpy(bias).cuda(), act, gated, dense, out=dense)
    check(dense, want, tol, f32)


@pytest.mark.gpu
@pytest.mark.parametrize("res32", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,M,K", [(70, 528, 1024), (261, 536, 640)])
def test_epilogue_of_aligned_rows(torch, T, M, K, gated, f32, res32):
    """Residuals and outputs whose rows start on 16 bytes, each with and without: loaded and stored whole, or not."""
    rng = np.random.default_rng(M + T)
    plan, x, xv, wv = make(torch, rng, T, M, K, "e2m1", False)
    mo = M // 2 if gated else M
    res = rng.standard_normal((T, mo)).astype(np.float32 if res32 else np.float16)
    want, tol = mx.product(xv, wv, None, "silu", gated, res)
    for gap, off in ((8, 8), (8, 1), (3, 0)):
        wide = torch.full((T, mo + gap), float("nan"), dtype=torch.float32 if res32 else torch.float16, device="cuda")
        r = wide[:, off:mo + off] if off + mo <= mo + gap else wide[:, :mo]
        r.copy_(torch.from_numpy(res))
        for ogap in (8, 1):
            out = torch.full((T + 1, mo + ogap), 7.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
            plan.run(x, act="silu", gated=gated, residual=r, out=out[:T, :mo])
            check(out[:T, :mo], want, tol, f32)
            assert (out[T] == 7).all() and (out[:, mo:] == 7).all()


# Counts from which, in one format or both, the library takes each of its kernels' tiles.
EVERY = [(18, 2054, 416), (33, 2054, 416), (33, 4106, 416), (33, 6002, 160), (50, 1100, 160), (50, 2054, 160), (70, 8202, 160),
         (100, 5130, 416), (129, 11010, 160), (129, 22018, 160), (193, 1000, 416), (193, 2054, 416), (257, 522, 160),
         (257, 2054, 416), (500, 28674, 416), (1001, 4106, 160)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,M,K", EVERY)
def test_every_kernel(torch, T, M, K, gated, fmt):
    rng = np.random.default_rng(M + T)
    plan, x, xv, wv = make(torch, rng, T, M, K, fmt, False)
    mo = M // 2 if gated else M
    bias = rng.standard_normal(M).astype(np.float32)
    res = rng.standard_normal((T, mo)).astype(np.float16)
    say(f"[gpu] product T {T} M {M} K {K} {fmt} gated {gated}")
    out = torch.full((T + 2, mo + 5), 7.0, device="cuda")
    y = out[1:1 + T, 2:2 + mo]
    plan.run(x, fmt, torch.from_numpy(bias).cuda(), "silu", gated, torch.from_numpy(res).cuda(), out=y)
    want, tol = mx.product(xv, wv, bias, "silu", gated, res)
    check(y, want, tol, True)
    edge = torch.ones_like(out, dtype=torch.bool)
    edge[1:1 + T, 2:2 + mo] = False
    assert (out[edge] == 7).all()


@pytest.mark.gpu
def test_nan_and_extreme_blocks(torch):
    """A NaN block reaches its own token's, or its own feature's, outputs only; the smallest exponents do not."""
    rng = np.random.default_rng(3)
    T, M, K = 20, 40, 256
    wc, we = weights(rng, M, K)
    we[7, 3] = 255
    we[9] = 0
    x = rng.standard_normal((T, K)).astype(np.float16)
    x[4, 100] = np.nan
    x[6] = 0
    plan = qmx.QMx(qmx.MxRows.pack(torch.from_numpy(mx.pack_bytes(wc, "e2m1")).cuda(), torch.from_numpy(we).cuda()))
    for fmt in FORMATS:
        y = plan.run(torch.from_numpy(x).cuda(), fmt, dtype=torch.float32).cpu().numpy()
        bad = np.zeros((T, M), dtype=bool)
        bad[4], bad[:, 7] = True, True
        assert np.array_equal(np.isnan(y), bad)
        assert (y[6, ~bad[6]] == 0).all()
        assert (np.abs(y[:, 9][~bad[:, 9]]) < 2.0 ** -100).all()


@pytest.mark.gpu
def test_streams_and_capture(torch):
    """Another stream, and a captured call that follows its inputs' contents over several replays."""
    rng = np.random.default_rng(5)
    for T, M, K, rows in [(1, 512, 1024, True), (16, 256, 4096, False), (40, 320, 2048, True), (300, 300, 512, True)]:
        plan, x, _, _ = make(torch, rng, T, M, K, "e2m1", rows)
        want = plan.run(x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = plan.run(x, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.run(x, out=out)
        for i in range(4):
            if rows:
                x.normal_()
            out.zero_()
            want = plan.run(x)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


@pytest.mark.gpu
def test_python_refusals(torch):
    w = qmx.quantize(torch.randn((32, 64), device="cuda"))
    plan = qmx.QMx(w)
    x = torch.randn((3, 64), device="cuda").half()
    for bad in (lambda: qmx.quantize(x.double()), lambda: qmx.quantize(x.t()), lambda: qmx.quantize(x, "e5m2"),
                lambda: qmx.quantize(x.cpu()), lambda: qmx.QMx(qmx.quantize(x, "e4m3")), lambda: plan.run(x[:, :32]),
                lambda: plan.run(x, act="tanh"), lambda: plan.run(x, residual=x), lambda: plan.run(x, dtype=torch.bfloat16),
                lambda: plan.run(x, bias=torch.zeros(31, device="cuda")), lambda: plan.run(x.cpu()),
                lambda: plan.run(x, out=torch.zeros((3, 16), device="cuda"), gated=False),
                lambda: w.values(torch.float64), lambda: qmx.MxRows.pack(x, x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qgemv.QgemvError):
        qmx.quantize(torch.randn((3, 48), device="cuda"))
    assert plan.run(x[:0]).shape == (0, 32) and qmx.quantize(x[:0]).values().shape == (0, 64)
