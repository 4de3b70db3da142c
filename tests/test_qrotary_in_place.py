"""q_out in q's place (qrotary_write): the same vectors, or refused, since lanes store where others still load."""

import pytest

from dense_sparse_bit_amd import qcache, qgemv, qrotary
from test_qrotary import freqs, i32


def refused(n_tok, heads, q, out):
    """Everything refused before a launch; the pointers are never followed."""
    kv = qcache.Rows(1 << 20, 0, 256, 128)
    r = qrotary._Rotary(128, 0, 1, 4096, None, None)
    st = qrotary.lib().qrotary_write(qcache.Shape(4, 2, 128, 64, 32), 4096, qcache.Seqs(n_tok, n_tok, 1, None, 4096, 4096), r, heads,
                                     q, out, kv, kv, None)
    return st == -1


@pytest.mark.parametrize("n_tok,heads,q,out", [
    (5, 3, (4096, 0, 384, 128), (4096, 1, 384, 128)),  # another type
    (5, 3, (4096, 1, 384, 128), (4096, 0, 384, 128)),
    (1, 1, (4096, 0, 384, 128), (4096, 1, 384, 128)),
    (5, 3, (4096, 0, 384, 128), (4096, 0, 392, 128)),  # other strides
    (5, 3, (4096, 0, 384, 128), (4096, 0, 512, 136)),
    (5, 3, (4096, 0, 0, 128), (4096, 0, 384, 128)),
    (5, 1, (4096, 0, 256, 128), (4096, 0, 128, 128)),
    (1, 3, (4096, 0, 384, 128), (4096, 0, 384, 256))])
def test_other_vectors_in_the_place_of_q(n_tok, heads, q, out):
    assert refused(n_tok, heads, qcache.Rows(*q), qcache.Rows(*out))


@pytest.mark.gpu
def test_in_place():
    """A stride that is of no account may differ; views of one stacked product are turned where they lie; the rest is refused."""
    import torch
    D, H = 64, 2
    c = qcache.QCache(4, H, D, page_size=16)
    r = qrotary.Rotary(freqs(D))
    k = torch.randn((3, H, D), device="cuda").half()
    pages, lens = i32(torch, [[0], [1], [2]]), i32(torch, [4, 9, 2])
    wide = torch.randn((3, 6, D), device="cuda").half()
    for q, n in ((wide[:, :4], 3), (wide[:1, :4], 1), (wide[:, :1], 3), (wide[:, ::2], 3)):
        want = r.write(c, q.clone(), k[:n], k[:n], lens[:n], pages[:n])
        assert torch.equal(r.write(c, q, k[:n], k[:n], lens[:n], pages[:n], out=q), want)
    one = wide[:1, :4]
    want = r.write(c, one.clone(), k[:1], k[:1], lens[:1], pages[:1])
    assert torch.equal(r.write(c, one, k[:1], k[:1], lens[:1], pages[:1], out=one.as_strided((1, 4, D), (8 * D, D, 1))), want)
    q = wide[:, :4]
    before = wide.clone()
    with pytest.raises(qgemv.QgemvError):
        r.write(c, q, k, k, lens, pages, out=wide.as_strided((3, 4, D), (4 * D, D, 1)))
    torch.cuda.synchronize()
    assert torch.equal(wide, before)
