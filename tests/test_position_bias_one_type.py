"""A table of two dimensions, one type, and its gradient of the same shape."""
import pytest
import torch

import window_gather_swin_gb300 as wgs

DEV = "cuda:0"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_gradient_of_a_two_dimensional_table(dtype):
    bucket = wgs.build_window_buckets((1, 4, 6))
    plan = wgs.build_bucket_plan(bucket, 77, device=DEV)
    gen = torch.Generator(DEV).manual_seed(1)
    table = torch.nn.Parameter(torch.randn(77, 4, generator=gen, device=DEV).to(dtype))
    grad = torch.randn(9, 4, 24, 24, generator=gen, device=DEV).to(dtype)
    assert wgs.position_bias(table.detach(), bucket.to(DEV)).shape == (1, 4, 24, 24)
    want = wgs.position_bias_bwd(grad, plan, dtype=dtype)
    assert want.shape == (1, 77, 4)
    out = torch.empty_like(table.detach())
    got = wgs.position_bias_bwd(grad, plan, dtype=dtype, grad_table=out)
    assert got is out and torch.equal(got, want[0])
    table.grad = got
    types = torch.zeros(9, dtype=torch.int32, device=DEV)
    for kw in ({"win_type": types, "n_types": 2}, {}):
        with pytest.raises(RuntimeError, match="shape"):
            wgs.position_bias_bwd(grad, plan, dtype=dtype, grad_table=out if kw else out[:76], **kw)
    wgs.check_error(DEV)
