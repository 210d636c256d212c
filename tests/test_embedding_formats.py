"""The formats that the embedding calls take from a given output."""
import pytest
import torch

import window_gather_swin_gb300 as wgs
from test_embedding import DEV, DT, FORMATS, _bits, _indices

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,tfmt", FORMATS)
@pytest.mark.parametrize("shape", [(90, 7, 40), (3000, 300, 24)], ids=str)
def test_a_given_output_names_the_format(shape, fmt, tfmt):
    n, rows, width = shape
    idx = _indices(n, rows, "skew", 1)
    grad = torch.randn(n, width, device=DEV).to(DT[fmt])
    own = torch.full((rows, width), float("nan"), dtype=DT[tfmt], device=DEV)
    got = wgs.embedding_bwd(grad, idx, rows, 0.7, grad_table=own)
    assert got is own and torch.equal(_bits(own), _bits(wgs.embedding_bwd(grad, idx, rows, 0.7, DT[tfmt])))
    out = torch.empty_like(grad)
    assert torch.equal(_bits(wgs.embedding(own, idx, 2.0, out=out)), _bits(wgs.embedding(own, idx, 2.0, DT[fmt])))
    # without one, float32; one of another format than `dtype` is refused
    assert wgs.embedding_bwd(grad, idx, rows).dtype is torch.float32
    for dtype, other in ((torch.float32, own.half()), (DT[fmt], own.double()), (None, own.double())):
        with pytest.raises(RuntimeError):
            wgs.embedding_bwd(grad, idx, rows, dtype=dtype, grad_table=other)
    with pytest.raises(RuntimeError, match="float32 or"):
        wgs.embedding_bwd(grad.bfloat16(), idx, rows, grad_table=own.half())
