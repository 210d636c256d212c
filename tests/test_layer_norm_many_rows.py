"""Layer norm's forward over more rows than a call's units have slots, so that slots
are filled and read again and units meet many times; and residual sums of tensors
that start at different places in 16 bytes.  Bounds as in test_layer_norm."""
import pytest
import torch

import window_gather_swin_gb300 as wgs
from test_layer_norm import DEV, _bits, _check_forward, _inputs, _same

pytestmark = pytest.mark.gpu

# at most 304 blocks of at most 4 units, of up to 4 slots each: every unit comes round
WIDE = [(9000, 1544), (8000, 2048), (6000, 2056), (6000, 4096), (3000, 6144), (2500, 7168), (3000, 8192), (2500, 8184)]
BESIDE = [("f16", 30000, 321), ("f32", 30000, 321), ("bf16", 8000, 1601), ("f16", 8000, 2041), ("bf16", 4000, 5201),
          ("f32", 6000, 2601), ("f32", 30000, 257), ("f16", 30000, 377)]


def _check(x, w, b, add):
    y, mean, rstd = wgs.layer_norm(x, w, b)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)
    total, y2, mean2, rstd2 = wgs.residual_add_layer_norm(x, add, w, b)
    assert torch.equal(_bits(total), _bits((x.float() + add.float()).to(x.dtype)))
    _check_forward(total, w, b, 1e-5, y2, mean2, rstd2)
    assert _same(wgs.layer_norm(total, w, b), (y2, mean2, rstd2))
    # in place, and again
    own, branch = x.clone(), add.clone()
    got = wgs.residual_add_layer_norm(own, branch, w, b, residual_out=own, out=branch)
    assert _same(got, (total, y2, mean2, rstd2))
    own = x.clone()
    assert _same(wgs.layer_norm(own, w, b, out=own), (y, mean, rstd))


@pytest.mark.parametrize("fmt,pfmt", [("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", WIDE, ids=str)
def test_many_wide_rows_of_16_bits(shape, fmt, pfmt):
    _check(*_inputs(*shape, fmt, pfmt, shape[1])[:3], _inputs(*shape, fmt, pfmt, 1)[4])


@pytest.mark.parametrize("fmt,rows,width", BESIDE)
def test_many_ragged_rows_with_two_blocks_beside(fmt, rows, width):
    _check(*_inputs(rows, width, fmt, "f32", width)[:3], _inputs(rows, width, fmt, "f32", 1)[4])


def test_many_wide_rows_replayed():
    """A captured call gives the eager call's bits, with new inputs written before
    each replay."""
    src = [_inputs(6000, 4096, "bf16", "bf16", k) for k in range(3)]
    x, w, b, _, add = (t.clone() for t in src[0])
    want = [wgs.residual_add_layer_norm(s[0], s[4], s[1], s[2]) for s in src]
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            got = wgs.residual_add_layer_norm(x, add, w, b)
        for s, ref in zip(src, want):
            for to, value in zip((x, w, b, add), (s[0], s[1], s[2], s[4])):
                to.copy_(value)
            graph.replay()
            torch.cuda.synchronize()
            assert _same(got, ref)


@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(10, 1), (9, 2), (6, 5), (8, 9), (257, 64), (41, 771), (3000, 96), (400, 192), (2500, 321),
                                   (30, 2050), (900, 2048), (500, 4096)], ids=str)
def test_residual_sums_of_views_that_start_anywhere(shape, fmt):
    """Each tensor its own number of elements into a buffer of NaN: element by element
    where they differ, in chunks where they are alike."""
    rows, width = shape
    x, w, b, _, add = _inputs(rows, width, fmt, "f32", 7)
    size = x.numel()
    total = (x.float() + add.float()).to(x.dtype)
    for starts in ((1, 2, 3, 4), (0, 1, 0, 0), (3, 0, 0, 5), (5, 5, 5, 5), (7, 7, 7, 6), (0, 0, 1, 1)):
        buf = torch.full((4, (size + 40) // 8 * 8), float("nan"), dtype=x.dtype, device=DEV)
        xv, av, tv, yv = (buf[i, 8 + at:8 + at + size].view(x.shape) for i, at in enumerate(starts))
        xv.copy_(x), av.copy_(add)
        got, y, mean, rstd = wgs.residual_add_layer_norm(xv, av, w, b, 1e-3, residual_out=tv, out=yv)
        assert got is tv and torch.equal(_bits(tv), _bits(total))
        _check_forward(total, w, b, 1e-3, y, mean, rstd)
        # in place of the inputs, which stay as they are where they are not outputs
        assert torch.equal(_bits(xv), _bits(x)) and torch.equal(_bits(av), _bits(add))
        again = wgs.residual_add_layer_norm(xv, av, w, b, 1e-3, residual_out=xv, out=av)
        assert torch.equal(_bits(again[0]), _bits(total))
        _check_forward(total, w, b, 1e-3, *again[1:])
        for i, at in enumerate(starts):
            assert buf[i, :8 + at].isnan().all() and buf[i, 8 + at + size:].isnan().all()
