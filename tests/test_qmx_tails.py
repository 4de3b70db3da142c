"""The MX product's activations: their own error, relative to their value, far below zero as well, and their ends.

x = 0 makes x W^T zero, so that what is activated is the bias, an fp32 number known exactly.  Bounds are those of
test_epilogue_tails for the forms that define the activations; the shorter forms here stay within them, in units of 2^-24:

  silu       exp2 1 ulp (2), its correction 1, the sum 1, the reciprocal 1 ulp (2), the product 1: 7 of 12
  gelu_tanh  the argument w by a square, a sum, a product and two constants: 5 |w| of 6 |w|, the rest as silu
  gelu       4e-7 (7) and a product, of 33 and more
"""

import numpy as np
import pytest

from dense_sparse_bit_amd import qmx
from gpu_checks import say
from test_epilogue_tails import bound, exact, points

pytestmark = pytest.mark.gpu

# rows by features that the library gives to: one token's kernel, rows quantised on the way, few outputs, many outputs
CALLS = [(1, 1026, False), (3, 1026, True), (40, 1026, False), (2000, 1026, False)]


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


def product(torch, T, bias, act, gated, fmt, rows):
    """act(bias), [T, outputs] in fp32, of a product of zeros."""
    K = 96
    plan = qmx.QMx(qmx.quantize(torch.randn((len(bias), K), device="cuda")))
    x = torch.zeros((T, K), dtype=torch.float16, device="cuda")
    y = plan.run(x if rows else qmx.quantize(x, fmt), fmt, torch.from_numpy(bias).cuda(), act, gated, dtype=torch.float32)
    y = y.cpu().numpy()
    assert np.array_equal(y, np.broadcast_to(y[:1], y.shape), equal_nan=True)
    return y[0]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,M,rows", CALLS)
def test_relative_error_of_the_activations(torch, T, M, rows, act, fmt):
    t = points(act, M)
    say(f"[gpu] MX tails T {T} M {M} {act} {fmt}")
    want, tol = exact(t.astype(np.float64), act), bound(t.astype(np.float64), act)
    got = product(torch, T, t, act, False, fmt, rows).astype(np.float64)
    assert (np.abs(got - want) / np.abs(want) / tol).max() <= 1
    # gated, by an up value that brings the tail into the output: one rounding more
    up = np.float32(1e6)
    both = np.stack([t[:M // 2], np.full(M // 2, up)], axis=1).ravel()
    want, tol = want[:M // 2] * float(up), tol[:M // 2] + 2.0 ** -24 * (1 + 2.0 ** -20)
    got = product(torch, T, both, act, True, fmt, rows).astype(np.float64)
    assert (np.abs(got - want) / np.abs(want) / tol).max() <= 1


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,M,rows", CALLS)
def test_activations_at_the_ends(torch, T, M, rows, act, fmt):
    """Far below zero 0, far above t itself, infinity infinite, NaN NaN; -infinity times 0 is NaN."""
    low, high = [-1e4, -1e12, -1e20, -3e38], [1e4, 1e12, 1.7e13, 1e20, 2.4e38, 3e38, np.inf]
    t = np.zeros(M, np.float32)
    n = len(low) + len(high)
    t[:n + 2] = low + high + [np.nan, -np.inf]
    say(f"[gpu] MX ends T {T} M {M} {act} {fmt}")
    got = product(torch, T, t, act, False, fmt, rows)
    assert np.all(got[:len(low)] == 0) and np.array_equal(got[len(low):n], t[len(low):n]) and np.isnan(got[n])
    assert (got[n + 1] == 0 if act == "relu" else np.isnan(got[n + 1])) and not got[n + 2:].any()
    # gated by 1
    both = np.stack([t[:M // 2], np.ones(M // 2, np.float32)], axis=1).ravel()
    assert np.array_equal(product(torch, T, both, act, True, fmt, rows), got[:M // 2], equal_nan=True)
