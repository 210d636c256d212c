"""The gradient of few indices into wide rows, whose columns belong to several
blocks: the sums by test_embedding's bounds, and what each block does besides
(zeros, the check of indices) once for all columns."""
import pytest
import torch

import window_gather_swin_gb300 as wgs
from test_embedding import DEV, DT, _bits, _check_gradient, _indices

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["uniform", "one", "skew", "none"])
@pytest.mark.parametrize("fmt,tfmt", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("shape", [(1000, 1, 2048), (1024, 300, 768), (1023, 3, 8192), (37, 2, 32768), (900, 7, 4099),
                                   (1, 5000, 1000), (513, 40, 257), (1024, 20, 516), (640, 33, 32767)], ids=str)
def test_gradient_of_few_indices_into_wide_rows(shape, fmt, tfmt, kind):
    n, rows, width = shape
    idx = _indices(n, rows, kind, 2)
    gen = torch.Generator(DEV).manual_seed(n)
    grad = torch.randn(n, width, generator=gen, device=DEV).to(DT[fmt])
    table = torch.full((rows, width), float("nan"), dtype=DT[tfmt], device=DEV)
    got = wgs.embedding_bwd(grad, idx, rows, 1.7, DT[tfmt], grad_table=table)
    _check_gradient(grad, idx, rows, 1.7, got)
    assert torch.equal(_bits(got), _bits(wgs.embedding_bwd(grad, idx, rows, 1.7, DT[tfmt])))
    # whole numbers: sums of at most 8 * 1024, exact in 32 bits
    whole = torch.randint(-8, 9, (n, width), generator=gen, device=DEV).to(DT[fmt])
    want = torch.zeros(rows, width, dtype=torch.float64, device=DEV)
    want.index_add_(0, idx[idx >= 0].long(), whole[idx >= 0].double())
    assert torch.equal(wgs.embedding_bwd(whole, idx, rows, 1.0, DT[tfmt]), want.float().to(DT[tfmt]))
    wgs.check_error(DEV)


def test_a_bad_index_and_views_of_wide_rows():
    n, rows, width = 300, 9, 2047
    idx = _indices(n, rows, "uniform", 4)
    buf = torch.full((n * width + 8,), float("nan"), dtype=torch.float16, device=DEV)
    grad = buf[3:3 + n * width].view(n, width)
    grad.copy_(torch.randn(n, width, device=DEV))
    out = torch.full((rows * width + 8,), 3.0, dtype=torch.float16, device=DEV)
    got = wgs.embedding_bwd(grad, idx, rows, 1.0, torch.float16, grad_table=out[5:5 + rows * width].view(rows, width))
    _check_gradient(grad, idx, rows, 1.0, got)
    assert (out[:5] == 3.0).all() and (out[5 + rows * width:] == 3.0).all()
    off = idx.clone()
    off[150] = rows
    pad = idx.clone()
    pad[150] = -1
    assert torch.equal(wgs.embedding_bwd(grad, off, rows), wgs.embedding_bwd(grad, pad, rows))
    with pytest.raises(wgs.WgsError, match="WGS_ERR_INDEX"):
        wgs.check_error(DEV)
    wgs.check_error(DEV)
