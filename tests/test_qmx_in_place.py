"""The residual in y's place (qmx_run): the same rows, or refused, since lanes store where others still load."""

import pytest

from dense_sparse_bit_amd import qgemv, qmx


def status(rows, gated=0, **kw):
    """Everything refused before a launch; the pointers are never followed."""
    e = qgemv.Epilogue()
    e.gated, e.residual = gated, 4096
    for k, v in kw.items():
        setattr(e, k, v)
    return qmx.lib().qmx_run(qmx.Shape(6, 64, 0), 4096, qmx.Input(1 << 20, rows, 0, -1, 0), 4096, e, None, 0, None)


@pytest.mark.parametrize("rows,kw", [
    (1, dict(y_type=1)), (1, dict(residual_type=1)), (3, dict(y_type=1)), (3, dict(residual_type=1, gated=1)),
    (3, dict(ldr=8)), (3, dict(ldy=8)), (3, dict(ldy=8, ldr=16)), (2, dict(gated=1, ldy=6)), (300, dict(ldr=7))])
def test_other_rows_in_the_place_of_y(rows, kw):
    assert status(rows, **kw) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 300])
def test_in_place(T):
    """The same rows, dense or wider; for one row a stride is of no account."""
    import torch
    plan = qmx.QMx(qmx.quantize(torch.randn((96, 256), device="cuda")))
    x = qmx.quantize(torch.randn((T, 256), device="cuda"))
    for dt in (torch.float16, torch.float32):
        wide = torch.randn((T, 128), device="cuda").to(dt)
        r = wide[:, 8:104]
        want = plan.run(x, residual=r.clone(), dtype=dt)
        if T > 1:
            before = wide.clone()
            with pytest.raises(qgemv.QgemvError):
                plan.run(x, residual=r, out=wide.as_strided((T, 96), (96, 1), 8))
            torch.cuda.synchronize()
            assert torch.equal(wide, before)
        assert torch.equal(plan.run(x, residual=r, out=r), want)
