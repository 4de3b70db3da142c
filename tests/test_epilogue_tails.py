"""The activations' own error, relative to their value, far below zero as well.

x = 0 makes W x zero, so that t is the bias, an fp32 number known exactly, and
fp32 outputs show the activation alone.  Bounds on |dy| / |y| in units of
2^-24 (a rounding to fp32), for the forms that y is defined by:

  silu       t / (1 + exp(-t)): exp 3 ulp (6), the sum 1, the quotient 2.5 ulp (5)
  gelu_tanh  t / (1 + exp(-w)), w = 2 sqrt(2/pi) t (1 + 0.044715 t^2): w is off by two
             constants and four roundings (6 of w, so 6 |w| of the exponential), the rest as silu
  gelu       t/2 erfc(z), z = -t / sqrt 2 off by 2 (its constant and a rounding), which erfc's
             condition 2 z^2 + 1 = t^2 + 1 (for t < 0; less above) multiplies; erfc 16 ulp (32), the product 1

The ranges end where a factor would leave fp32's normal range.
"""

import math

import numpy as np
import pytest

from dense_sparse_bit_amd import qgemv
from gpu_checks import say
from test_epilogue import weights

LOWEST = {"silu": -85.0, "gelu_tanh": -9.5, "gelu": -12.5}


def wide(t):
    """The argument of gelu_tanh's exponential."""
    return 2 * math.sqrt(2 / math.pi) * t * (1 + 0.044715 * t * t)


def exact(t, act):
    """act(t) in fp64 without cancellation."""
    if act == "gelu":
        return 0.5 * t * np.array([math.erfc(-z / math.sqrt(2)) for z in t])
    return t / (1 + np.exp(-(wide(t) if act == "gelu_tanh" else t)))


def bound(t, act):
    units = {"silu": lambda: 12 + 0 * t, "gelu_tanh": lambda: 6 * np.abs(wide(t)) + 12,
             "gelu": lambda: 2 * (t * t + 1) + 33}[act]()
    return units * 2.0 ** -24


def points(act, n):
    lo = LOWEST[act]
    t = np.concatenate([np.linspace(lo, 12, n - 8), [-1e-6, 1e-6, -6.0, -5.5, -5.0, 0.5, 30.0, 1e4]])
    return t.astype(np.float32)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_sums_that_cancel_break_the_bound(act):
    """fp32 with a correctly rounded erf or tanh: 1 + erf and 1 + tanh miss the bound by far, the forms above keep it."""
    t = points(act, 400)
    f = np.float32
    z = t.astype(np.float64)
    if act == "gelu":
        bad = f(0.5) * t * (f(1) + np.array([math.erf(x / math.sqrt(2)) for x in z]).astype(f))
        good = f(0.5) * t * np.array([math.erfc(x) for x in (t * f(-0.70710678)).astype(np.float64)]).astype(f)
    else:
        bad = f(0.5) * t * (f(1) + np.tanh(wide(z) / 2).astype(f))
        good = t / (f(1) + np.exp(-(f(1.5957691) * (t * (f(1) + f(0.044715) * t * t)))))
    rel = lambda y: np.abs(y.astype(np.float64) - exact(z, act)) / np.abs(exact(z, act)) / bound(z, act)
    assert rel(bad).max() > 1e3
    assert rel(good).max() <= 1


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


# every place that applies the epilogue: k_stream, k_pair, k_split, k_xlds, k_huff
@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("name,M,K,batch", [("mlp7b_lut3", 1026, 96, 1), ("mlp70b_lut4", 1026, 96, 1),
                                            ("block7b_u3", 1026, 1024, 8), ("mlp7b_lut3", 8194, 96, 8),
                                            ("mlp7b_hptq", 258, 128, 1)])
def test_relative_error_of_the_activations(torch, name, M, K, batch, act):
    plan = qgemv.QGemv(weights(name, M, K))
    x = torch.zeros((batch, K), dtype=torch.float16, device="cuda")
    t = points(act, M)
    say(f"[gpu] epilogue tails {name} {M}x{K} batch {batch} {act}")
    got = plan.run_epilogue(x, bias=torch.from_numpy(t).cuda(), act=act, dtype=torch.float32)
    t64 = t.astype(np.float64)
    want, tol = exact(t64, act), bound(t64, act)
    err = np.abs(got.cpu().numpy().astype(np.float64) - want) / np.abs(want)
    assert float((err / tol).max()) <= 1, f"worst at t = {t[np.unravel_index((err / tol).argmax(), err.shape)[1]]}"
    # gated, by an up value that brings the tail into the output: one rounding more
    up = np.float32(1e6)
    both = np.stack([t[:M // 2], np.full(M // 2, up)], axis=1).ravel()
    got = plan.run_epilogue(x, bias=torch.from_numpy(both).cuda(), act=act, gated=True, dtype=torch.float32)
    want, tol = want[:M // 2] * float(up), tol[:M // 2] + 2.0 ** -24 * (1 + 2.0 ** -20)
    err = np.abs(got.cpu().numpy().astype(np.float64) - want) / np.abs(want)
    assert float((err / tol).max()) <= 1
    plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_at_the_ends(torch, act):
    """Far below zero 0, far above t itself, infinity infinite, NaN NaN."""
    M, K = 18, 96
    plan = qgemv.QGemv(weights("mlp7b_lut3", M, K))
    t = np.zeros(M, np.float32)
    t[:10] = [-1e4, -1e12, -1e20, -3e38, 1e4, 1e12, 1e20, 3e38, np.inf, np.nan]
    say(f"[gpu] epilogue ends {act}")
    x = torch.zeros((1, K), dtype=torch.float16, device="cuda")
    got = plan.run_epilogue(x, bias=torch.from_numpy(t).cuda(), act=act, dtype=torch.float32).cpu().numpy()[0]
    plan.close()
    assert np.all(got[:4] == 0) and np.array_equal(got[4:9], t[4:9]) and np.isnan(got[9]) and not got[10:].any()
