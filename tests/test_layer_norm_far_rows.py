"""Gradients of rows of one large value: what lies outside a row in its chunks takes
no part, whatever the row's mean and rstd.

A row of 2^121 has the distances 0, so h = 0 and grad_x = rstd (g - M(g)), far inside
FP32's range; mean rstd = 2^121 316 is not.  The statistics are given as the forward
would write them (eps 1e-5), so test_layer_norm's bounds hold.
"""
import pytest
import torch

import window_gather_swin_gb300 as wgs
from test_layer_norm import DEV, _bits, _check_backward, _inputs, _same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(5, 3), (300, 24), (40, 72), (33, 193), (700, 200), (41, 771), (12, 1000), (9, 4100),
                                        (7, 8184)])
def test_gradients_of_rows_of_one_large_value(rows, width, fmt):
    x, w, b, gy, past = _inputs(rows, width, fmt, "f32", rows)
    far = torch.arange(rows, device=DEV) % 3 == 1
    x[far] = 2.0 ** 121
    xd = x.double()
    mean = xd.mean(1)
    rstd = ((xd - mean[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    mean = mean.float()
    assert (mean[far] == 2.0 ** 121).all() and (mean * rstd).isinf().equal(far)
    for weight, residual in ((w, None), (w, past), (None, past)):
        got = wgs.layer_norm_bwd(gy, x, mean, rstd, weight, residual)
        assert not any(t.isnan().any() for t in got if t is not None)
        _check_backward(gy, x, mean, rstd, weight, residual, got)


@pytest.mark.parametrize("shift", [1, 3])
def test_of_views_and_beside_other_rows(shift):
    """The same at other places in memory, and other rows' bits as without such rows."""
    rows, width = 77, 200
    x, w, b, gy, past = _inputs(rows, width, "f32", "f32", 3)
    _, mean, rstd = wgs.layer_norm(x, w, b)
    want = wgs.layer_norm_bwd(gy, x, mean, rstd, w, past)[0]
    x[50], mean[50] = 2.0 ** 121, 2.0 ** 121
    rstd[50] = 316.0
    gx = wgs.layer_norm_bwd(gy, x, mean, rstd, w, past)[0]
    keep = torch.arange(rows, device=DEV) != 50
    assert _same((gx[keep],), (want[keep],)) and not gx.isnan().any()
    buf = torch.full((3, rows * width + 16), float("nan"), device=DEV)
    xv, gv, ov = (t[shift:shift + rows * width].view(rows, width) for t in buf)
    xv.copy_(x), gv.copy_(gy)
    got = wgs.layer_norm_bwd(gv, xv, mean, rstd, w, past, grad_x=ov)
    _check_backward(gy, x, mean, rstd, w, past, got)
