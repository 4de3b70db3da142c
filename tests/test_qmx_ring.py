"""The waits of the MX product's tile kernel (csrc/qmx_ring.h): a chunk has landed in LDS before it is read.

The CPU tests replay a wave's memory operations in their order.  A step's wait leaves the last N of them on the way; all copies
of the chunk that is read next must be among the others.
"""

import os
import shutil
import subprocess

import pytest

from dense_sparse_bit_amd import qmx
from gpu_checks import say

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_sparse_bit_amd", "csrc")
PROGRAM = """
#include <cstdio>
#include "qmx_ring.h"
int main() {
  int s, c, e, j;
  while (std::scanf("%d %d %d %d", &s, &c, &e, &j) == 4) std::printf("%d\\n", qmx_ring::may_be_on_the_way(s, c, e, j));
}
"""
# stages, copies of a chunk, operations for a quad's exponents of the kernel's tiles
E2M1 = [(8, 2, 4), (5, 3, 6), (4, 4, 8), (3, 6, 12)]
E4M3 = [(5, 3, 4), (4, 4, 6), (2, 8, 12)]


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    """{(stages, copies, exponents, j): N}"""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", CSRC, str(d / "ring.cpp"), "-o", str(d / "ring")], check=True)
    keys = [(s, c, e, j) for s, c, x in E2M1 + E4M3 for e in (0, x) for j in range(4)]
    out = subprocess.run([str(d / "ring")], input="\n".join(" ".join(map(str, k)) for k in keys), capture_output=True, text=True,
                         check=True).stdout
    return dict(zip(keys, map(int, out.split())))


def read_too_early(wait, stages, copies, exps, chunks, exponents_first):
    """The chunks that are read before they have landed.  wait(j, whether the step's quad issues exponents): N."""
    issued, early = [], []

    def landed(chunk, n):
        return all(op != chunk for op in issued[len(issued) - n:])

    issued += ["e"] * exps + [c for c in range(stages) for _ in range(copies)]
    if not landed(0, (stages - 1) * copies):
        early.append(0)
    for c in range(chunks):
        q, j = divmod(c, 4)
        more = q < chunks // 4  # the last, shorter quad needs no further exponents
        if c + 1 < chunks and not landed(c + 1, wait(j, more)):
            early.append(c + 1)
        ops = [[c + stages] * copies, ["e"] * exps if j == 0 and more else []]
        issued += sum(ops[::-1] if exponents_first else ops, [])
    return early


@pytest.mark.parametrize("exponents_first", [False, True])
@pytest.mark.parametrize("stages,copies,exps", E2M1 + E4M3)
def test_every_chunk_has_landed(waits, stages, copies, exps, exponents_first):
    for chunks in range(1, 30):
        wait = lambda j, more: waits[stages, copies, exps if more else 0, j]  # noqa: E731
        assert not read_too_early(wait, stages, copies, exps, chunks, exponents_first), chunks


@pytest.mark.parametrize("stages,copies,exps", [t for t in E2M1 + E4M3 if t[0] > 2])
def test_counting_exponents_that_are_not_issued_is_too_early(waits, stages, copies, exps):
    """With three chunks in the last quad the third would be read before it is there.  (Of eight stages only where these are
    all: otherwise the quad before has issued exponents behind the third.)"""
    wait = lambda j, more: waits[stages, copies, exps, j]  # noqa: E731
    early = [n for n in range(1, 30) if read_too_early(wait, stages, copies, exps, n, False)]
    assert early == (list(range(3, 30, 4)) if stages < 8 else [3])


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
# rows by features that the library gives, in one format or both, to each of the kernel's tiles
SIZES = [(257, 2054), (64, 22018), (2000, 8202), (1001, 4106), (4100, 8200), (500, 28674)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("K", [320, 384, 864, 1408, 2432])
@pytest.mark.parametrize("T,M", SIZES)
def test_three_chunks_in_the_last_quad(T, M, K, fmt):
    """Every output, three times: blocks of which the last chunk's are the largest."""
    import torch
    say(f"[gpu] product T {T} M {M} K {K} {fmt}")
    w = qmx.quantize(torch.randn((M, K), device="cuda"))
    size = torch.ones(K, device="cuda")
    size[-(K % 128 or 128):] = 16
    x = qmx.quantize(torch.randn((T, K), device="cuda") * size, fmt)
    plan, xv, wv = qmx.QMx(w), x.values().double(), w.values().double()
    want = xv @ wv.t()
    tol = ((128 + K / 128 + 16) * 2.0 ** -24 + 2.0 ** -24) * (xv.abs() @ wv.abs().t()) + 2.0 ** -126  # and the output's rounding
    for _ in range(3):
        assert ((plan.run(x, dtype=torch.float32).double() - want).abs() <= tol).all()
