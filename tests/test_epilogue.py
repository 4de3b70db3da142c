"""The quantized product with its epilogue (qgemv_run_epilogue) against the oracle.

t = W x + bias, y = act(t) + residual, or act(t[2i]) * t[2i + 1] + residual.
Two references per case:

* the fp64 oracle.  dt <= 1e-4 A + 1e-6 is the products' own tolerance; it goes
  through act with |act'| <= 1.13 (gelu's largest slope; silu's is 1.10), and
  through the gate's product.
* qgemv_run's fp32 sums, through the epilogue in fp64.  The sums are the same,
  so only the epilogue's own roundings count: the bias add 2^-24 |t|, a few
  fp32 roundings inside act (its factors are formed to about an ulp and, where
  1 + erf or 1 + tanh cancels, to an ulp of 1: at most 2^-21 (|t| + 1) in all),
  the gate's product and the residual add 2^-24 each, and the rounding to FP16
  (eps/2 = 2^-11 of the value, 2^-25 where it is subnormal).
"""

import ctypes
import math

import numpy as np
import pytest

from dense_sparse_bit_amd import qgemv
from gpu_checks import CANARY, say
from oracle import gemv, pack
from synth import make_format_inputs

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
SLOPE = 1.13


def act64(t, act):
    if act == "relu":
        return np.maximum(t, 0)
    if act == "gelu":
        return t * np.vectorize(lambda z: 0.5 * math.erfc(-z / math.sqrt(2)))(t)
    if act == "gelu_tanh":
        return t * 0.5 * (1 + np.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
    if act == "silu":
        return t * np.exp(-np.logaddexp(0, -t))
    return t


def weights(name, M, K):
    f = make_format_inputs(name, 0, M, K)
    counts = np.bincount(f["rows"], minlength=f["M"])
    f["row_ptr"] = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    f["col_idx"] = f["cols"].astype(np.int32)
    return f


# ---------------------------------------------------------------------------
# CPU
# ---------------------------------------------------------------------------
def test_library_exports_the_entry_point():
    assert hasattr(qgemv.lib(), "qgemv_run_epilogue")


def test_null_arguments_are_refused_before_any_gpu_call():
    e = qgemv.Epilogue()
    f = qgemv.lib().qgemv_run_epilogue
    assert f(None, 16, 16, 1, ctypes.byref(e), None) == -1
    assert f(16, None, 16, 1, ctypes.byref(e), None) == -1
    assert f(16, 16, None, 1, ctypes.byref(e), None) == -1


@pytest.mark.parametrize("name,M,K", [("block7b_u3", 19, 256), ("tiny_u4", 5, 64), ("mlp7b_lut3", 18, 160),
                                      ("mlp70b_lut4", 7, 96), ("mlp7b_bpdq3", 6, 192)])
def test_interleave_rows_alternates_both_weight_sets(name, M, K):
    a, b = weights(name, M, K), weights(name, M + 1, K)
    for key in ("codes_packed", "scales", "zeros", "lut", "coefs"):
        if key in b:
            b[key] = b[key][:M]
    b["M"] = M
    n = int(b["row_ptr"][M])
    b["row_ptr"], b["col_idx"], b["values"] = b["row_ptr"][:M + 1], b["col_idx"][:n], b["values"][:n]
    w = qgemv.interleave_rows(a, b)
    assert w["M"] == 2 * M
    D = gemv.decode(w) + gemv.sparse_dense(w)
    assert np.array_equal(D[0::2], gemv.decode(a) + gemv.sparse_dense(a))
    assert np.array_equal(D[1::2], gemv.decode(b) + gemv.sparse_dense(b))
    codes = qgemv.unpack_host(qgemv.repack(w), 2 * M, K)  # the repacker takes it as valid
    assert np.array_equal(codes[0::2], pack.unpack_bitstream(a["codes_packed"], a["bits"], K))


def test_interleave_rows_refuses_unlike_sets():
    a = weights("tiny_u4", 4, 64)
    with pytest.raises(ValueError):
        qgemv.interleave_rows(a, weights("block7b_u3", 4, 64))
    with pytest.raises(ValueError):
        qgemv.interleave_rows(a, weights("tiny_u4", 5, 64))
    h = weights("mlp7b_hptq", 2, 128)
    with pytest.raises(ValueError):
        qgemv.interleave_rows(h, h)


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


_PLANS = {}


@pytest.fixture(scope="module")
def plans(torch):
    def get(name, M, K):
        if (name, M, K) not in _PLANS:
            w = weights(name, M, K)
            x = np.random.default_rng(M + K).standard_normal((16, K)).astype(np.float16)
            y, A = gemv.gemv(w, x)
            _PLANS[name, M, K] = (qgemv.QGemv(w), x, y, A)
        return _PLANS[name, M, K]
    yield get
    for p in _PLANS.values():
        p[0].close()
    _PLANS.clear()


def check(torch, got, t32, t64, dt, act, gated, bias, res, what):
    """got against both references (see the module's text); t32 / t64: the sums W x of qgemv_run and the oracle."""
    half = got.dtype == torch.float16
    g = got.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(g)), f"{what}: output not fully written"
    b = 0.0 if bias is None else bias.cpu().numpy().astype(np.float64)
    r = 0.0 if res is None else res.cpu().numpy().astype(np.float64)
    for name, t, d in (("oracle", t64, dt), ("qgemv_run", t32, np.zeros_like(dt))):
        t = t + b
        d = d + 2.0 ** -24 * np.abs(t)
        if gated:
            a, u = act64(t[:, 0::2], act), t[:, 1::2]
            da = SLOPE * d[:, 0::2] + 2.0 ** -21 * (np.abs(t[:, 0::2]) + 1)
            v = a * u
            dv = da * np.abs(u) + np.abs(a) * d[:, 1::2] + da * d[:, 1::2] + 2.0 ** -24 * np.abs(v)
        else:
            v = act64(t, act)
            dv = SLOPE * d + 2.0 ** -21 * (np.abs(t) + 1) * (act != "none")
        y = v + r
        dv = dv + 2.0 ** -24 * np.abs(y)
        tol = dv + (2.0 ** -11 * (np.abs(y) + dv) + 2.0 ** -25 if half else 0) + 1e-30
        err = np.abs(g - y)
        worst = float((err / tol).max())
        assert worst <= 1, f"{what} against {name}: worst error is {worst:.2f} of the tolerance"


# every kernel family: k_stream batch 1 (one and two blocks a chunk), k_pair, k_split, k_xlds, k_stream batch 8/16, k_huff
SHAPES = [("block7b_u3", 34, 2080), ("tiny_u4", 98, 512), ("mlp7b_lut3", 34, 4128), ("mlp70b_lut4", 24, 8192),
          ("mlp7b_bpdq3", 66, 2112), ("mlp7b_hptq", 34, 1024), ("mlp7b_lut3", 8194, 256), ("block7b_u3", 8210, 192),
          ("mlp70b_lut4", 4370, 160), ("block7b_u3", 2, 32), ("mlp7b_lut3", 34, 11008)]


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 8, 16])
@pytest.mark.parametrize("name,M,K", SHAPES)
def test_formats_batches_and_gates(torch, plans, name, M, K, batch):
    plan, x16, y64, A = plans(name, M, K)
    x = torch.from_numpy(x16[:batch]).cuda()
    t64, dt = y64[:batch], 1e-4 * A[:batch] + 1e-6
    t32 = plan.run(x).cpu().numpy().astype(np.float64)
    gen = torch.Generator(device="cuda").manual_seed(M * K + batch)
    for i, (gated, act) in enumerate([(False, "gelu"), (True, "silu"), (False, "none"), (True, "relu")]):
        mo = M // 2 if gated else M
        bt, rt, yt = [(torch.float16, torch.float32, torch.float16), (torch.float32, torch.float16, torch.float32),
                      (None, torch.float16, torch.float16), (torch.float16, None, torch.float32)][i]
        bias = torch.randn(M, generator=gen, device="cuda").to(bt) if bt else None
        res = torch.randn((batch, mo), generator=gen, device="cuda").to(rt) if rt else None
        say(f"[gpu] epilogue {name} {M}x{K} batch {batch} act {act} gated {gated} y {yt}")
        out = torch.full((batch, mo), float("nan"), dtype=yt, device="cuda")
        got = plan.run_epilogue(x, bias=bias, act=act, gated=gated, residual=res, out=out)
        assert got is out
        check(torch, got, t32, t64, dt, act, gated, bias, res, f"{name} {M}x{K} b{batch} {act}")
        again = plan.run_epilogue(x, bias=bias, act=act, gated=gated, residual=res, dtype=yt)
        assert torch.equal(got, again), "not bitwise deterministic"


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("name,M,K,batch", [("mlp7b_lut3", 33, 96, 1), ("tiny_u4", 33, 96, 8)])
def test_activations_over_their_range(torch, plans, name, M, K, batch, act):
    """Odd M; biases that put t from far below zero to far above it."""
    plan, x16, y64, A = plans(name, M, K)
    x = torch.from_numpy(x16[:batch]).cuda()
    t32 = plan.run(x).cpu().numpy().astype(np.float64)
    bias = torch.linspace(-120, 120, M, device="cuda")
    say(f"[gpu] epilogue activation {act} batch {batch}")
    got = plan.run_epilogue(x, bias=bias, act=act, dtype=torch.float32)
    # a bias of up to 120 leaves |t| 2^-24 in the sum: counted in check()
    check(torch, got, t32, y64[:batch], 1e-4 * A[:batch] + 1e-6, act, False, bias, None, act)


@pytest.mark.gpu
@pytest.mark.parametrize("name,M,K,batch", [("block7b_u3", 98, 512, 16), ("mlp7b_bpdq3", 98, 512, 8),
                                            ("mlp70b_lut4", 98, 512, 1)])
@pytest.mark.parametrize("gated", [False, True])
def test_strided_rows_and_residual_in_place(torch, plans, name, M, K, batch, gated):
    """y as columns of a wider array, framed by canaries; then y += product in place."""
    plan, x16, y64, A = plans(name, M, K)
    x = torch.from_numpy(x16[:batch]).cuda()
    t32 = plan.run(x).cpu().numpy().astype(np.float64)
    mo = M // 2 if gated else M
    wide = torch.empty((batch + 2, mo + 37), dtype=torch.float32, device="cuda")
    wide.view(torch.int32).fill_(int(CANARY))
    out = wide[1:batch + 1, 5:5 + mo]
    say(f"[gpu] epilogue strided {name} batch {batch} gated {gated}")
    plan.run_epilogue(x, act="silu", gated=gated, out=out)
    check(torch, out, t32, y64[:batch], 1e-4 * A[:batch] + 1e-6, "silu", gated, None, None, "strided")
    mask = torch.ones_like(wide, dtype=torch.bool)
    mask[1:batch + 1, 5:5 + mo] = False
    assert torch.all(wide.view(torch.int32)[mask] == int(CANARY)).item(), "a write landed outside y"
    base = torch.randn((batch, mo + 3), device="cuda").half()
    res = base[:, 2:2 + mo]
    before = res.clone()
    plan.run_epilogue(x, gated=gated, residual=res, out=res)
    check(torch, res, t32, y64[:batch], 1e-4 * A[:batch] + 1e-6, "none", gated, None, before, "in place")


@pytest.mark.gpu
@pytest.mark.parametrize("name,M,K,batch", [("block7b_u3", 130, 1024, 16), ("mlp7b_lut3", 130, 1024, 1)])
def test_captured_and_on_another_stream(torch, plans, name, M, K, batch):
    plan, x16, _, _ = plans(name, M, K)
    xs = [torch.from_numpy(np.ascontiguousarray(np.roll(x16[:batch], k, axis=1))).cuda() for k in range(3)]
    res = torch.randn((batch, M), device="cuda").half()
    want = [plan.run_epilogue(x, act="gelu", residual=res).clone() for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    say(f"[gpu] epilogue on a side stream and captured, batch {batch}")
    got = plan.run_epilogue(xs[1], act="gelu", residual=res, stream=s)
    s.synchronize()
    assert torch.equal(got, want[1])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = plan.run_epilogue(x, act="gelu", residual=res)
    for k in (2, 0, 1, 1):
        x.copy_(xs[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])
        assert torch.equal(plan.run_epilogue(xs[2], act="gelu", residual=res), want[2])


@pytest.mark.gpu
def test_refusals(torch, plans):
    plan, x16, _, _ = plans("tiny_u4", 33, 96)
    x = torch.from_numpy(x16[:1]).cuda()
    y = torch.zeros((1, 33), device="cuda")
    L = qgemv.lib()

    def call(batch=1, x=x, y=y, off=0, **kw):
        e = qgemv.Epilogue()
        e.y_type = 1
        for k, v in kw.items():
            setattr(e, k, v)
        return L.qgemv_run_epilogue(plan._h, x.data_ptr() + off, y.data_ptr(), batch, ctypes.byref(e),
                                    torch.cuda.current_stream().cuda_stream)

    assert L.qgemv_run_epilogue(plan._h, x.data_ptr(), y.data_ptr(), 1, None, None) == -1
    assert call(batch=2) == -3 and call(batch=0) == -3 and call(batch=-1) == -3
    assert call(act=5) == -3 and call(act=-1) == -3
    assert call(y_type=2) == -3 and call(bias_type=-1) == -3 and call(residual_type=7) == -3
    assert call(gated=1) == -3  # M is odd
    assert call(ldy=32) == -1 and call(ldr=-1) == -1
    assert call(off=2) == -1
    assert call(bias=y.data_ptr() + 1) == -1 and call(residual=y.data_ptr() + 2, residual_type=1) == -1
    for bad in (lambda: plan.run_epilogue(x.float()), lambda: plan.run_epilogue(x[:, :64]),
                lambda: plan.run_epilogue(x, act="tanh"), lambda: plan.run_epilogue(x, dtype=torch.bfloat16),
                lambda: plan.run_epilogue(x, bias=torch.zeros(32, device="cuda")),
                lambda: plan.run_epilogue(x, bias=torch.zeros(33)),
                lambda: plan.run_epilogue(x, residual=torch.zeros((1, 34), device="cuda")),
                lambda: plan.run_epilogue(x, out=torch.zeros((1, 66), device="cuda")[:, ::2]),
                lambda: plan.run_epilogue(x, out=y, dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qgemv.QgemvError):
        plan.run_epilogue(x, gated=True)
    torch.cuda.synchronize()
    assert torch.all(y == 0).item()
