"""Where the sums over a row's waves lie in LDS (csrc/qnorm_sums.h), and the norms whose sums are of two types.

A wave may write its part of a sum while a slower one still reads the parts of the sum before, so the bytes of consecutive
sums must be disjoint, whatever their types.  Between a sum and the next but one lies a barrier that every wave reaches after its
reads.
"""

import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest

from dense_sparse_bit_amd import qnorm
from gpu_checks import say
from oracle import block
from test_qnorm import check, data

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_sparse_bit_amd", "csrc")
PROGRAM = """
#include <cstdio>
#include "qnorm_sums.h"
int main() {
  std::printf("%d\\n", qnorm_sums::kBytes);
  for (int at = 0, i = 0; i < 8; ++i) std::printf("%d\\n", at = qnorm_sums::next(at));
}
"""


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    """(bytes, offsets of a row's first sums)"""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("sums")
    (d / "sums.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", CSRC, str(d / "sums.cpp"), "-o", str(d / "sums")], check=True)
    n, *at = map(int, subprocess.run([str(d / "sums")], capture_output=True, text=True, check=True).stdout.split())
    return n, at


def sums(layer, post, wide):
    """Bytes of a part of each of a row's sums: the post norm's are fp32, the other's fp32 or, wide, 64 bits."""
    one = 2 if layer else 1
    return (one * [4] if post else []) + one * [8 if wide else 4]


@pytest.mark.parametrize("waves", [2, 4, 8, 16])
def test_consecutive_sums_share_no_byte(layout, waves):
    n, at = layout
    for layer, post, wide in itertools.product([False, True], repeat=3):
        ranges = [range(o, o + waves * size) for o, size in zip(at, sums(layer, post, wide))]
        for r in ranges:
            assert 0 <= r.start and r.stop <= n and r.start % 16 == 0
        for a, b in zip(ranges, ranges[1:]):
            assert a.stop <= b.start or b.stop <= a.start, (layer, post, wide, a, b)


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm GPU"
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,N", [(200, 4128), (256, 8192), (300, 8224), (300, 16384), (60, 32768)])
def test_sixteen_waves_a_row(torch, T, N, kind):
    """Both norms with sixteen waves a row, into fp32 and into blocks, every row of them."""
    say(f"[gpu] both norms {T}x{N} {kind}")
    a, g = data(torch, T, N, N + T)
    kw = dict(post="post", gate="gate", pre="pre")
    (h, dh), (o, do) = block.norm(a["y"], a["h"], **{k: a[v] for k, v in kw.items()}, kind=kind)
    call = lambda out: qnorm.norm(g["y"], g["h"], **{k: g[v] for k, v in kw.items()}, kind=kind, out_type=out)  # noqa: E731
    got_h, got = call("fp32")
    check(got_h, h, dh, "h")
    check(got, o, do, "out")
    most = np.repeat(np.abs(o).reshape(T, -1, 32).max(2) + do.reshape(T, -1, 32).max(2), 32, axis=1)
    # half an element's step: 2^-2 or 2^-4 of the value, at least half the smallest element, which is below 1/12 or 2^-17 of
    # the block's largest value
    for fmt, part, least in (("e2m1", 2.0 ** -2, 1 / 12), ("e4m3", 2.0 ** -4, 2.0 ** -17)):
        got_h, got = call(fmt)
        check(got_h, h, dh, "h")
        v = got.values().cpu().numpy().astype(np.float64)
        assert (np.abs(v - o) <= np.maximum(part * (np.abs(o) + do), least * most) + do).all(), fmt
