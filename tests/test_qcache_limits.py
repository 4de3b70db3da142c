"""The largest calls of qcache_write and qcache_read: a launch of 256 threads a workgroup has fewer than 2^24 workgroups."""

import numpy as np
import pytest

from dense_sparse_bit_amd import qcache, qgemv
from gpu_checks import say
from oracle import cache as oc


def workgroups(n_seq, n_tok, heads, start):
    units = n_tok // 16 + 2 * n_seq if start else n_seq
    return (units + 1) // 2 * heads


# (n_seq, n_tok, heads, with q_start): one row each, prompts, many heads
PAST = [(2**20, 2**20, 32, False), (2**20 - 1, 2**20 - 1, 32, False), (2**10 + 1, 2**10 + 1, 65535, False),
        (1, 2**25, 16, True), (2**24, 1, 1, True), (2**28, 2**28, 1, False), (1, 2**31 - 1, 65535, True)]


@pytest.mark.parametrize("n_seq,n_tok,heads,start", PAST)
def test_calls_past_a_launch_refused(n_seq, n_tok, heads, start):
    """Refused before a launch; the pointers are never followed."""
    assert workgroups(n_seq, n_tok, heads, start) * 256 >= 2**32
    sh, rows = qcache.Shape(4, heads, 64, 64, 32), qcache.Rows(4096, 0, 0, 0)
    sq = qcache.Seqs(n_seq, n_tok, 1, 4096 if start else None, 4096, 4096)
    for f in (qcache.lib().qcache_write, qcache.lib().qcache_read):
        assert f(sh, 4096, sq, rows, rows, None) == -3


@pytest.mark.gpu
def test_largest_launch():
    """2^20 - 2 one-row sequences of 32 heads, nearly all on no page, and one more pair of sequences refused."""
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    S, H, D = 2**20 - 2, 32, 64
    assert workgroups(S, S, H, False) * 256 < 2**32 <= workgroups(S + 2, S + 2, H, False) * 256
    c = qcache.QCache(2, H, D, page_size=16)
    c.data.zero_()
    lens = torch.ones(S + 2, dtype=torch.int32, device="cuda")
    pages = torch.full((S + 2, 1), -1, dtype=torch.int32, device="cuda")
    pages[S - 1], pages[0] = 1, 0
    row = torch.randn((1, H, D), device="cuda").half()
    k = row.expand(S + 2, H, D)
    say("[gpu] cache write, 2^20 - 2 sequences x 32 heads")
    c.write(k[:S], k[:S], lens[:S], pages[:S])
    got = c.read(lens[:2], torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"), dtype=torch.float32)
    want = oc.held(row.cpu().numpy(), 32).astype(np.float32)
    for g in got:
        assert np.array_equal(g.cpu().numpy(), np.broadcast_to(want, g.shape))
    with pytest.raises(qgemv.QgemvError) as e:
        c.write(k, k, lens, pages)
    assert e.value.status == -3
