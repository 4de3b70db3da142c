"""h' in FP16 beside fp32 rows or blocks is rounded once: what lies next to the middle between two FP16 numbers goes to its side."""

import numpy as np
import pytest

from dense_sparse_bit_amd import qnorm
from gpu_checks import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


@pytest.mark.parametrize("out", ["fp32", "e2m1", "e4m3"])
@pytest.mark.parametrize("T,N", [(1, 64), (5, 1024), (530, 4096), (3, 8192), (2, 32768)])
def test_stream_in_fp16_is_rounded_once(torch, T, N, out):
    """h' = y + 2^-30 h, exact in 64 bits.  y is the middle between two FP16 numbers, or just any fp32 number."""
    rng = np.random.default_rng(N)
    m = rng.integers(1024, 2048, (T, N))
    y = ((2 * m + 1) * 2.0 ** rng.integers(-14, 4, (T, N)) * rng.choice([-1, 1], (T, N)) / 1024).astype(np.float32)
    y[:, ::3] = rng.standard_normal(y[:, ::3].shape)
    h = rng.integers(-2, 3, (T, N)).astype(np.float16)
    want = (y.astype(np.float64) + 2.0 ** -30 * h.astype(np.float64)).astype(np.float16)
    say(f"[gpu] norm, stream in FP16, {T}x{N} {out}")
    got, _ = qnorm.norm(torch.from_numpy(y).cuda(), torch.from_numpy(h).cuda(), scale=2.0 ** -30,
                        pre=torch.ones(N, device="cuda"), out_type=out)
    assert got.dtype == torch.float16
    assert np.array_equal(got.cpu().numpy(), want)
