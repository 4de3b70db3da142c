"""bench.py --step-ctx: the bytes it counts, and a short run of the step it times."""

import numpy as np
import pytest

import bench


def test_step_bytes_counts_every_operand_once():
    w = {}
    for name, M, K in (("qkv", 96, 32), ("o", 32, 32), ("gate_up", 128, 32), ("down", 32, 64)):
        nnz = M
        w[name] = {"M": M, "K": K, "bits": 3, "fmt": "uniform", "group": 16,
                   "row_ptr": np.arange(M + 1, dtype=np.int32) * (nnz // M)}
    B, ctx = 2, 10
    weights = sum(x["M"] * x["K"] * 3 // 8 + x["M"] * (x["K"] // 16) * 4 + 6 * x["M"] + 4 * (x["M"] + 1)
                  for x in w.values())
    inputs = sum(2 * B * x["K"] for x in w.values())
    outputs = 2 * B * (96 + 32 + 64 + 32)  # gate_up's output is one value per row pair
    E = bench.HEADS_7B * bench.HEAD_DIM_7B
    cache = B * (ctx + 1) * 2 * bench.HEADS_7B * (64 + 16)
    assert bench.step_bytes(w, B, ctx, 32) == weights + inputs + outputs + cache + 2 * B * (3 * E + E + 2 * E)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 16])
def test_step_runs(batch):
    """measure_step checks that the step's outputs are finite and the same for every weight copy."""
    import torch

    from dense_sparse_bit_amd import qgemv
    dev = torch.device("cuda:0")
    ms, alg, copies = bench.measure_step(torch, qgemv, batch, 100, 3, 1, 0.0, torch.cuda.Stream(device=dev), dev, True)
    assert ms > 0 and copies == 2 and alg > 100_000_000
