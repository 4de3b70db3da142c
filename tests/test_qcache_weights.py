"""What qcache_attend's weights and sums hold, seen through values that show them.

The weights are two FP16 parts each (22 bits), the values FP16, everything else
fp32.  Over random values the output's own rounding to FP16 hides most of that,
so here

* two nearly equal weights stand on values +V and -V: the output is V tanh of
  half their distance, small, with a small rounding, and V times any error of
  a weight stays in it;
* every block of 128 positions has its own dimension and size of value, so that
  a block lost, doubled or taken from elsewhere changes one output by more
  than a tenth of it;
* the error of random outputs is held in the 2-norm, against the same
  arithmetic in numpy.
"""

import math

import numpy as np
import pytest

from dense_sparse_bit_amd import qcache
from gpu_checks import say
from oracle import cache as oc
from test_qcache import Batch, fill

D, G = 128, 32


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


def rounded_attend(q, k, v, scale, parts):
    """One row [Hq, D] over held k, v [L, H, D]: fp64 but for the values and the output in FP16, and weights
    2^7 above the largest's in `parts` FP16 parts."""
    per = q.shape[0] // k.shape[1]
    out = np.empty(q.shape)
    for h in range(q.shape[0]):
        s = scale * math.log2(math.e) * (k[:, h // per] @ q[h].astype(np.float64))
        p = np.exp2(s - s.max() + 7)
        w = np.zeros_like(p)
        for _ in range(parts):
            w += (p - w).astype(np.float16)
        out[h] = (w @ v[:, h // per].astype(np.float16).astype(np.float64)) / p.sum()
    return out.astype(np.float16).astype(np.float64)


# ---- the weights' second part ---------------------------------------------------
V, STEP, HEADS, PER = 1.5, 2.0 ** -6, 2, 16


def pair(L, at):
    """Keys and values of positions `at` and at + 1 (of one tile); the others lie 47 and more below them, on zeros."""
    k, v = np.zeros((L, HEADS, D), np.float16), np.zeros((L, HEADS, D), np.float16)
    k[:, :, 0] = -60000
    k[at, :, 0], k[at + 1, :, 0] = 0, 1
    v[at], v[at + 1] = V, -V
    q = np.zeros((1, HEADS * PER, D), np.float16)
    q[0, :, 0] = np.linspace(0.05, 1, HEADS * PER)
    return k, v, q


def pair_tolerance(want):
    """In units of 2^-24: a weight is exp2(7 - distance) with its exponent rounded twice (2 x 7 ln 2 = 9.7), off by
    2^-18 of the scores, which are 2^-6 (1), exp2 an ulp (2), its two parts 2^-22 (4); sums and products 4: 21 of V,
    and as much of the small output.  Then the output's rounding."""
    return V * 2.0 ** -19 + 2.0 ** -11 * np.abs(want) + 2.0 ** -25


CASES = [(2, 0), (1000, 500), (1000, 14), (1000, 998)]


@pytest.mark.parametrize("L,at", CASES)
def test_one_part_would_be_seen(L, at):
    k, v, q = pair(L, at)
    hk, hv = oc.held(k, G), oc.held(v, G)
    want = oc.attend(q, hk, hv, STEP, [L - 1])[0][0]
    assert np.abs(want).max() < V * 2.0 ** -6
    err = {n: float((np.abs(rounded_attend(q[0], hk, hv, STEP, n) - want) / pair_tolerance(want)).max()) for n in (1, 2)}
    assert err[1] > 4 and err[2] <= 1, err


@pytest.mark.gpu
@pytest.mark.parametrize("L,at", CASES)
def test_weights_hold_22_bits(torch, L, at):
    k, v, q = pair(L, at)
    b = Batch(torch, [L], [1], 64, seed=L, one_each=True)
    c, enc = fill(torch, b, HEADS, D, G, seed=0, keys=lambda s, _: k, vals=lambda s, _: v)
    want = oc.attend(q, *[oc.values(e) for e in enc[0]], STEP, [L - 1])[0]
    say(f"[gpu] attend two nearly equal weights at {at} of {L}")
    got = c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=STEP).cpu().numpy().astype(np.float64)
    assert float((np.abs(got - want) / pair_tolerance(want)).max()) <= 1


# ---- every block ----------------------------------------------------------------
def blocks(L, seed):
    """Values: block b of 128 positions holds 4 + b // D in dimension b % D and nothing elsewhere."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((L, 1, D)).astype(np.float16)
    v = np.zeros((L, 1, D), np.float16)
    b = np.arange(L) // 128
    v[np.arange(L), 0, b % D] = 4 + b // D
    q = rng.standard_normal((1, 4, D)).astype(np.float16)
    q[:, 0] = 0  # equal weights
    return k, v, q


def block_tolerance(q, k, want, scale, L):
    """All values are positive, so relative to the output: values and output 2^-11, weights 2^-22, exp2 2^-22, scores as
    in test_qcache ((2^-18 + 2^-23) B), numerator and denominator each; fp32 sums (L / 32 + 16) 2^-24 each; and weights
    below FP16's range, 2^-32 of the largest each, times the largest value."""
    e = oc.quantise(k, G)
    B = scale * (np.abs(q[0].astype(np.float64)) @ oc.reach(e)[:, 0].T).max(axis=1)[:, None]
    rel = 2 * 2.0 ** -11 + 2 * ((2.0 ** -18 + 2.0 ** -23) * B + 2 * 2.0 ** -22) + 2 * (L / 32 + 16) * 2.0 ** -24
    return rel * np.abs(want) + L * 2.0 ** -32 * 9 + 2.0 ** -25


@pytest.mark.parametrize("L", [16384, 70000])
def test_a_lost_block_would_be_seen(L):
    k, v, q = blocks(L, L)
    hk, hv, scale = oc.held(k, G), oc.held(v, G), 1 / math.sqrt(D)
    want = oc.attend(q, hk, hv, scale, [L - 1])[0][0]
    tol = block_tolerance(q, k, want, scale, L)
    for h in range(q.shape[1]):
        s = scale * (hk[:, 0] @ q[0, h].astype(np.float64))
        p = np.exp(s - s.max())
        for b in range(-(-L // 128)):
            part = p[128 * b:128 * b + 128] @ hv[128 * b:128 * b + 128, 0, b % D] / p.sum()
            assert part > 4 * tol[h, b % D]


@pytest.mark.gpu
@pytest.mark.parametrize("L,page", [(16384, 16), (70000, 64)])
def test_every_block_counts(torch, L, page):
    k, v, q = blocks(L, L)
    scale = 1 / math.sqrt(D)
    b = Batch(torch, [L], [1], page, seed=L, one_each=True)
    c, enc = fill(torch, b, 1, D, G, seed=0, keys=lambda s, _: k, vals=lambda s, _: v)
    want = oc.attend(q, *[oc.values(e) for e in enc[0]], scale, [L - 1])[0][0]
    say(f"[gpu] attend, a value per block, L={L} page={page}")
    got = c.attend(torch.from_numpy(q).cuda(), *b.args(), scale=scale).cpu().numpy()[0].astype(np.float64)
    assert float((np.abs(got - want) / block_tolerance(q, k, want, scale, L)).max()) <= 1


# ---- the error over all outputs ---------------------------------------------------
def random_row(L, seed):
    rng = np.random.default_rng(seed)
    k, v = (rng.standard_normal((L, 2, D)).astype(np.float16) for _ in range(2))
    return k, v, rng.standard_normal((1, 16, D)).astype(np.float16)


def norm_error(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


def norms(L):
    """The outputs exactly, and the 2-norms of the error with one and with two parts (3.3 and 2.7, 3.5 and 2.9e-4)."""
    k, v, q = random_row(L, L)
    hk, hv, scale = oc.held(k, G), oc.held(v, G), 1 / math.sqrt(D)
    want = oc.attend(q, hk, hv, scale, [L - 1])[0][0]
    return want, *(norm_error(rounded_attend(q[0], hk, hv, scale, n), want) for n in (1, 2))


@pytest.mark.parametrize("L", [150, 3000])
def test_norms_of_one_and_two_parts_differ(L):
    _, one, two = norms(L)
    assert one > 1.15 * two


@pytest.mark.gpu
@pytest.mark.parametrize("L", [150, 3000])
def test_norm_of_the_outputs_error(torch, L):
    k, v, q = random_row(L, L)
    b = Batch(torch, [L], [1], 64, seed=L, one_each=True)
    c, _ = fill(torch, b, 2, D, G, seed=0, keys=lambda s, _: k, vals=lambda s, _: v)
    want, one, two = norms(L)
    say(f"[gpu] attend, 2-norm of the error, L={L}")
    e = norm_error(c.attend(torch.from_numpy(q).cuda(), *b.args()).cpu().numpy()[0].astype(np.float64), want)
    assert e < math.sqrt(one * two), f"{e:.3e}: one part has {one:.3e}, two have {two:.3e}"
