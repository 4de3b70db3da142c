"""Pairs whose axis positions do not have are left as they are, whatever they hold (qrotary_write)."""

import numpy as np
import pytest

from dense_sparse_bit_amd import qcache, qrotary
from gpu_checks import say
from test_qrotary import check_turned, freqs, i32, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("style", ["halves", "neighbours"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 96), (256, 256)])
def test_pairs_of_no_axis_stay(torch, D, rot, style, f32):
    """Infinities, NaN and both zeros in them reach neither their partners nor anything else."""
    rng = np.random.default_rng(D + rot)
    T, H, lens = 37, 2, [5, 32]
    ty = np.float32 if f32 else np.float16
    axis = rng.integers(-1, 3, rot // 2)  # -1 and 2 are none of the two axes
    pos = rng.integers(-1000, 2 ** 20, (2, T)).astype(np.int32)
    q, k, v = (rng.standard_normal((T, n, D)).astype(ty) for n in (5, H, H))
    first = np.arange(rot // 2) if style == "halves" else 2 * np.arange(rot // 2)
    second = first + (rot // 2 if style == "halves" else 1)
    stay = np.flatnonzero((axis < 0) | (axis > 1))
    for x in (q, k):
        for t in range(T):
            i = stay[t % len(stay)]
            x[t, 0, first[i]] = [np.inf, -np.inf, np.nan, -0.0][t % 4]
            x[t, 1, second[i]] = [np.nan, -0.0, np.inf, -np.inf][t % 4]
            x[t, 1, first[i]] = -1.0
    own = np.concatenate([first[stay], second[stay], np.arange(rot, D)])
    turned = np.setdiff1d(np.arange(D), own)
    f = freqs(rot)
    pages, total = table(torch, lens, 16)
    gq, gk, gv = (torch.from_numpy(a).cuda() for a in (q, k, v))
    r = qrotary.Rotary(f, style, axis)
    args = (i32(torch, lens), pages, i32(torch, [0, 5, 37]))
    say(f"[gpu] rotary, pairs of no axis, D {D} rot {rot} {style} {ty.__name__}")

    def check(got, x):
        got = got.cpu().numpy()
        with np.errstate(over="ignore"):
            want = x[..., own].astype(got.dtype)
        assert np.array_equal(got[..., own], want, equal_nan=True)
        zero = want == 0
        assert np.array_equal(np.signbit(got[..., own][zero]), np.signbit(want[zero]))
        assert np.isfinite(got[..., turned]).all()

    c = qcache.QCache(total, H, D, page_size=16)
    for dt in (torch.float16, torch.float32):
        out = r.write(c, gq, gk, gv, *args, positions=i32(torch, pos), out=torch.empty_like(gq, dtype=dt))
        check(out, q)
    finite = np.where(np.isfinite(q), q, 0)
    check_turned(r.write(c, torch.from_numpy(finite).cuda(), gk, gv, *args, positions=i32(torch, pos)), finite, pos, f, style, axis)
    # the cache holds of the keys what it holds of the same keys turned as queries
    tk = r.write(c, gk, gk, gv, *args, positions=i32(torch, pos))
    check(tk, k)
    one, two = (qcache.QCache(total, H, D, page_size=16) for _ in range(2))
    one.data.zero_()
    two.data.zero_()
    r.write(one, None, gk, gv, *args, positions=i32(torch, pos))
    two.write(tk, gv.half(), *args)
    assert torch.equal(one.data, two.data)
