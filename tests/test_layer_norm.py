"""Layer norm with weight and bias, fused with a residual add, and its
gradients, against the formulas in double precision.

Tolerances, with u = 2^-24 and D = 32 a bound on the additions that a value of
a row's sum passes through (a thread's 16 columns in pairs: 8; its pair: 1; the
lanes of a warp: 5; the warps of a unit: 16), X and S the row's largest |x| and
|x - mean|:

* the rounded mean that distances are taken from is off by e = (D + 2) u X, so
  distances are at most S' = S + e and each is off by u S' from rounding;
* mean: |err| <= (D + 3) u S' + u |mean|;
* the variance is a mean of squares of at most S'^2 less the square of the
  distances' mean: off by (D + 8) u (var + e^2); rstd, relatively, by half of
  that over var + eps, and 2u: R;
* h = (x - mean) rstd: |err| <= rstd (2 u S' + err of the distances' mean) +
  |h| (R + 2u); y = h w + b adds |w| times that and u |y|;
* gradients, given mean and rstd: h is off by 3u relatively, g = gy w by u, the
  means by (D + 6) u of their terms' magnitudes, so grad_x by (D + 12) u of
  rstd (|g| + M|g| + |h| M|g h|) (+ |grad_residual|);
* columns' sums: a thread's rows (at most rows / 152 and a tile of 8), the rows
  of a warp (2), the units of a block (16), the blocks (5 + 5): (rows / 152 +
  48) u of the sum of the terms' magnitudes;
* rounding to the output's format adds half a step (half a subnormal step at
  the bottom).
"""
import math

import pytest
import torch

import oracle
import window_gather_swin_gb300 as wgs
from window_gather_swin_gb300 import _capi

DEV = "cuda:0"
U, D = 2.0 ** -24, 32
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OK, NULL, SHAPE, WIDTH, ALIGN, DTYPE, ARCH, LAUNCH, INDEX, ALIAS = range(10)
PTR = [0x10000000 * k for k in range(1, 14)]


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def _same(a, b):
    return all((p is None and q is None) or torch.equal(_bits(p), _bits(q)) for p, q in zip(a, b))


def _half_step(want, dtype):
    f = torch.finfo(dtype)
    return want.abs().clamp(min=f.smallest_normal) * (f.eps / 2)


# --------------------------------------------------------------- formulas ----

def _formulas(x, w, b, eps):
    xd = x.double()
    mean = xd.mean(-1, keepdim=True)
    var = (xd - mean).square().mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    return mean, var, rstd, (xd - mean) * rstd * w + b


def _gradients(gy, x, mean, rstd, w):
    h = (x - mean) * rstd
    g = gy * w
    gx = rstd * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    return gx, (gy * h).sum(0), gy.sum(0)


def test_formulas_equal_torch_and_the_oracle():
    gen = torch.Generator().manual_seed(1)
    x, w, b = torch.randn(6, 10, generator=gen), torch.randn(10, generator=gen), torch.randn(10, generator=gen)
    mean, _, rstd, y = _formulas(x, w.double(), b.double(), 1e-5)
    want = torch.nn.functional.layer_norm(x.double(), (10,), w.double(), b.double(), 1e-5)
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-12)
    oy, om, orr = oracle.group_norm_act(x.numpy()[:, None], 1, w.double().numpy(), b.double().numpy(), 1e-5, None,
                                        "f32")
    assert torch.allclose(y, torch.from_numpy(oy)[:, 0], rtol=1e-12, atol=1e-12)
    assert torch.allclose(mean, torch.from_numpy(om), rtol=1e-12, atol=1e-14)
    assert torch.allclose(rstd, torch.from_numpy(orr), rtol=1e-12)


def test_gradient_formulas_equal_differences():
    """Central differences of sum(gy y) + sum(past x) in double: error O(step^2)
    + noise / step, both far below 1e-7 at a step of 1e-5."""
    gen = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x, gy, past, w, b = rand(3, 7), rand(3, 7), rand(3, 7), rand(7), rand(7)
    mean, _, rstd, _ = _formulas(x, w, b, 1e-3)
    gx, gw, gb = _gradients(gy, x, mean, rstd, w)

    def value(args):
        return ((_formulas(*args, 1e-3)[3] * gy).sum() + (past * args[0]).sum()).item()

    for which, grad in ((0, gx + past), (1, gw), (2, gb)):
        for i in range(grad.numel()):
            args = [x.clone(), w.clone(), b.clone()]
            args[which].view(-1)[i] += 1e-5
            up = value(args)
            args[which].view(-1)[i] -= 2e-5
            assert abs((up - value(args)) / 2e-5 - grad.view(-1)[i].item()) < 1e-7


# --------------------------------------------------------------- refusals ----

def test_layer_norm_refusals():
    """Every call here is refused while its arguments are checked."""
    lib = _capi.load()
    x, w, b, y, m, r = PTR[:6]

    def call(x=x, w=w, b=b, y=y, m=m, r=r, rows=100, width=64, dtype=1, param=0):
        return lib.layer_norm(x, w, b, y, m, r, rows, width, 1e-5, dtype, param, None)

    assert call(dtype=3) == DTYPE and call(dtype=-1) == DTYPE and call(param=2) == DTYPE
    assert call(dtype=0, param=1) == DTYPE
    assert call(width=0) == WIDTH and call(width=-4) == WIDTH and call(width=8193) == WIDTH
    assert call(rows=-1) == SHAPE and call(rows=2 ** 60) == SHAPE
    assert call(x=None, y=None, rows=0) == OK
    assert call(x=None) == NULL and call(y=None) == NULL and call(w=None) == NULL
    assert call(m=None) == NULL and call(r=None) == NULL
    assert call(x=x + 1) == ALIGN and call(y=y + 1) == ALIGN and call(w=w + 2) == ALIGN
    assert call(b=b + 1) == ALIGN and call(m=m + 2) == ALIGN and call(x=x + 2, dtype=0) == ALIGN
    assert call(y=x + 64) == ALIAS and call(y=w) == ALIAS and call(m=r) == ALIAS and call(m=x + 32) == ALIAS
    assert call(r=b) == ALIAS and call(m=y + 128) == ALIAS


def test_residual_add_layer_norm_refusals():
    lib = _capi.load()
    a, c, w, b, t, y, m, r = PTR[:8]

    def call(a=a, c=c, w=w, b=b, t=t, y=y, m=m, r=r, rows=100, width=64, dtype=2, param=2):
        return lib.residual_add_layer_norm(a, c, w, b, t, y, m, r, rows, width, 1e-5, dtype, param, None)

    for name in ("a", "c", "t", "y", "w", "m"):
        assert call(**{name: None}) == NULL, name
    assert call(c=c + 1) == ALIGN and call(t=t + 1) == ALIGN
    assert call(t=y) == ALIAS and call(t=a + 64) == ALIAS and call(y=c + 2) == ALIAS and call(t=y + 64) == ALIAS
    assert call(t=a, y=a) == ALIAS
    assert call(a=None, c=None, t=None, y=None, rows=0) == OK


def test_layer_norm_bwd_refusals():
    lib = _capi.load()
    gy, x, m, r, w, past, gx, gw, gb, ws = PTR[:10]
    need = lib.wgs_layer_norm_bwd_workspace_bytes(100, 64)
    assert need > 0 and lib.wgs_layer_norm_bwd_workspace_bytes(0, 64) == 0
    assert lib.wgs_layer_norm_bwd_workspace_bytes(-1, 64) == 0
    assert lib.wgs_layer_norm_bwd_workspace_bytes(100, 8193) == 0

    def call(gy=gy, x=x, m=m, r=r, w=w, past=past, gx=gx, gw=gw, gb=gb, ws=ws, size=need, rows=100, width=64,
             dtype=1, param=0):
        return lib.layer_norm_bwd(gy, x, m, r, w, past, gx, gw, gb, ws, size, rows, width, dtype, param, None)

    assert call(dtype=7) == DTYPE and call(param=2) == DTYPE
    assert call(width=0) == WIDTH and call(width=9000) == WIDTH
    assert call(rows=-1) == SHAPE and call(size=need - 1) == SHAPE
    for name in ("gy", "x", "m", "r", "gx", "ws"):
        assert call(**{name: None}) == NULL, name
    assert call(gy=None, x=None, gx=None, gw=None, gb=None, ws=None, rows=0) == OK
    assert call(gy=gy + 1) == ALIGN and call(past=past + 1) == ALIGN and call(ws=ws + 8) == ALIGN
    assert call(gw=gw + 2) == ALIGN and call(r=r + 1) == ALIGN
    for over in (dict(gx=x + 64), dict(gx=gy + 64), dict(gx=past + 2), dict(gw=w), dict(gw=gb), dict(ws=x + 64),
                 dict(gx=w), dict(ws=m), dict(gb=r), dict(ws=past), dict(ws=gx + 16)):
        assert call(**over) == ALIAS, over


def test_python_refuses_cpu_tensors():
    x = torch.zeros(3, 8)
    for call in (lambda: wgs.layer_norm(x), lambda: wgs.residual_add_layer_norm(x, x),
                 lambda: wgs.layer_norm_bwd(x, x, torch.zeros(3), torch.zeros(3))):
        with pytest.raises(RuntimeError, match="CUDA"):
            call()
    assert wgs.layer_norm_bwd_workspace_bytes(100, 64) > 0
    with pytest.raises(RuntimeError, match="at most"):
        wgs.layer_norm_bwd_workspace_bytes(100, 2 ** 31)


# -------------------------------------------------------------------- GPU ----

SHAPES = [  # rows, width: every unit, both ends of its widths, whole and odd chunks
    (1, 1), (300, 1), (3, 2), (9, 5), (1, 32), (700, 16), (33, 33), (100, 64), (61, 90), (2500, 96), (50, 97),
    (31, 128), (7, 129), (144, 192), (5000, 192), (1000, 193), (45, 252), (46, 255), (20, 257), (257, 384),
    (39, 385), (26, 512), (27, 511), (24, 516), (65, 771), (700, 768), (40, 1024), (33, 1536), (17, 1537), (9, 2050),
    (12, 2048), (5, 4097), (400, 4100), (3, 8192), (320, 8191), (2, 6144), (1, 7000),
]
FORMATS = [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")]


def _inputs(rows, width, fmt, pfmt, seed, offset=1.0):
    gen = torch.Generator(DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    x = (rand(rows, width) * (0.5 + torch.rand(width, generator=gen, device=DEV)) + offset * rand(width)).to(DT[fmt])
    return (x, (1 + 0.2 * rand(width)).to(DT[pfmt]), (0.2 * rand(width)).to(DT[pfmt]),
            rand(rows, width).to(DT[fmt]), rand(rows, width).to(DT[fmt]))


def _check_forward(x, w, b, eps, y, mean, rstd):
    wd = torch.ones(x.shape[1], device=DEV).double() if w is None else w.double()
    bd = torch.zeros_like(wd) if b is None else b.double()
    eps = torch.tensor(eps).double().item()
    m, var, r, want = _formulas(x, wd, bd, eps)
    xd = x.double()
    far = (D + 2) * U * xd.abs().amax(1, keepdim=True)
    S = (xd - m).abs().amax(1, keepdim=True) + far
    tol_d = (D + 3) * U * S                      # of the distances' mean
    assert ((mean.double()[:, None] - m).abs() <= tol_d + U * m.abs()).all()
    R = 0.5 * (D + 8) * U * (var + far * far) / (var + eps) + 2 * U
    assert ((rstd.double()[:, None] - r).abs() <= R * r).all()
    h = ((xd - m) * r).abs()
    tol = (r * (2 * U * S + tol_d) + h * (R + 2 * U)) * wd.abs() + U * want.abs()
    tol = tol * (1 + torch.finfo(x.dtype).eps) + _half_step(want, x.dtype)
    err = (y.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()


def _check_backward(gy, x, mean, rstd, w, past, got):
    gx, gw, gb = got
    rows, width = x.shape
    wd = torch.ones(width, device=DEV).double() if w is None else w.double()
    md, rd, xd, gd = mean.double()[:, None], rstd.double()[:, None], x.double(), gy.double()
    want, want_w, want_b = _gradients(gd, xd, md, rd, wd)
    h, g = ((xd - md) * rd).abs(), (gd * wd).abs()
    mag = rd * (g + g.mean(1, keepdim=True) + h * (g * h).mean(1, keepdim=True))
    if past is not None:
        want = want + past.double()
        mag = mag + past.double().abs()
    tol = (D + 12) * U * mag * (1 + torch.finfo(x.dtype).eps) + _half_step(want, x.dtype)
    err = (gx.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    if w is None:
        assert gw is None and gb is None
        return
    for v, ref, size in ((gw, want_w, (gd.abs() * h).sum(0)), (gb, want_b, gd.abs().sum(0))):
        tol = (rows / 152 + 48) * U * size * (1 + torch.finfo(w.dtype).eps) + _half_step(ref, w.dtype)
        err = (v.double() - ref).abs()
        assert v.dtype == w.dtype and (err <= tol).all(), (err / tol).max()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,pfmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer_norm_and_gradients(shape, fmt, pfmt):
    rows, width = shape
    x, w, b, gy, add = _inputs(rows, width, fmt, pfmt, rows + width)
    y, mean, rstd = wgs.layer_norm(x, w, b, 1e-5)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)
    # the residual form: the rounded sum, and the norm of that, bit for bit
    total, y2, mean2, rstd2 = wgs.residual_add_layer_norm(x, add, w, b, 1e-5)
    assert torch.equal(_bits(total), _bits((x.float() + add.float()).to(x.dtype)))
    assert _same(wgs.layer_norm(total, w, b, 1e-5), (y2, mean2, rstd2))
    need = wgs.layer_norm_bwd_workspace_bytes(rows, width)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)    # NaN patterns
    got = wgs.layer_norm_bwd(gy, x, mean, rstd, w, workspace=ws)
    _check_backward(gy, x, mean, rstd, w, None, got)
    past = wgs.layer_norm_bwd(gy, x, mean, rstd, w, add, workspace=ws)
    _check_backward(gy, x, mean, rstd, w, add, past)
    assert (ws[need:] == 0xff).all()
    # the workspace's contents do not matter, and the same call gives the same bits
    assert _same(wgs.layer_norm_bwd(gy, x, mean, rstd, w, add), past)
    wgs.check_error(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(333, 192), (41, 771), (12, 2050), (3, 8192)], ids=str)
def test_outputs_in_place_of_inputs(shape, fmt):
    x, w, b, gy, add = _inputs(*shape, fmt, "f32", 5)
    y, mean, rstd = wgs.layer_norm(x, w, b)
    own = x.clone()
    wgs.layer_norm(own, w, b, out=own)
    assert _same((own,), (y,))
    want = wgs.residual_add_layer_norm(x, add, w, b)
    for t_in, y_in in ((0, 1), (1, 0), (0, None), (None, 0), (None, 1)):
        given = [x.clone(), add.clone()]
        got = wgs.residual_add_layer_norm(*given, w, b, residual_out=None if t_in is None else given[t_in],
                                          out=None if y_in is None else given[y_in])
        assert _same(got, want)
    want = wgs.layer_norm_bwd(gy, x, mean, rstd, w, add)
    for k in range(3):
        given = [gy.clone(), x.clone(), add.clone()]
        got = wgs.layer_norm_bwd(given[0], given[1], mean, rstd, w, given[2], grad_x=given[k])
        assert _same(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (2, 3), (257, 64), (5, 771), (3000, 96), (30, 2050)], ids=str)
def test_views_that_start_anywhere(shape, fmt):
    """Tensors that each start a different number of elements into a buffer, with
    and without weights; what lies around them stays."""
    rows, width = shape
    x, w, b, gy, add = _inputs(rows, width, fmt, "f32", 7)
    size, pad = x.numel(), 40
    buf = torch.full((6, size + 2 * pad), 3.0, dtype=x.dtype, device=DEV)
    for shift in (1, 2, 3, 4, 7):
        buf.fill_(3.0)
        at = [pad + (shift * (i + 1)) % 8 for i in range(6)]
        xv, gv, av, yv, tv, gxv = (buf[i, at[i]:at[i] + size].view(x.shape) for i in range(6))
        xv.copy_(x), gv.copy_(gy), av.copy_(add)
        y, mean, rstd = wgs.layer_norm(xv, None, None, 1e-3, out=yv)
        _check_forward(x, None, None, 1e-3, y, mean, rstd)
        total, y, mean, rstd = wgs.residual_add_layer_norm(xv, av, w, None, 1e-3, residual_out=tv, out=yv)
        _check_forward(total, w, None, 1e-3, y, mean, rstd)
        got = wgs.layer_norm_bwd(gv, tv, mean, rstd, w, av, grad_x=gxv)
        _check_backward(gy, total, mean, rstd, w, add, got)
        none = wgs.layer_norm_bwd(gv, tv, mean, rstd, grad_x=gxv)
        _check_backward(gy, total, mean, rstd, None, None, none)
        for i in range(6):
            assert (buf[i, :at[i]] == 3.0).all() and (buf[i, at[i] + size:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (2, 3), (5, 8), (9, 20), (257, 64), (13, 771), (2000, 96), (30, 2050),
                                   (5, 1536), (3, 8190)], ids=str)
def test_views_that_all_start_at_the_same_place(shape, fmt):
    """All tensors the same number of elements into 16 bytes: rows are read in chunks
    that begin before the first one.  With fewer rows than lanes and units take, and
    with more."""
    rows, width = shape
    x, w, b, gy, add = _inputs(rows, width, fmt, "f32", 7)
    size, pad = x.numel(), 40
    want = wgs.residual_add_layer_norm(x, add, w, b)
    for shift in range(1, 8):
        buf = torch.full((6, (size + 2 * pad) // 8 * 8), 3.0, dtype=x.dtype, device=DEV)
        at = 8 + shift
        xv, gv, av, yv, tv, gxv = (buf[i, at:at + size].view(x.shape) for i in range(6))
        xv.copy_(x), gv.copy_(gy), av.copy_(add)
        y, mean, rstd = wgs.layer_norm(xv, w, b, 1e-5, out=yv)
        _check_forward(x, w, b, 1e-5, y, mean, rstd)
        total, y, mean, rstd = wgs.residual_add_layer_norm(xv, av, w, b, residual_out=tv, out=yv)
        assert _same((total,), want[:1])
        _check_forward(total, w, b, 1e-5, y, mean, rstd)
        got = wgs.layer_norm_bwd(gv, tv, mean, rstd, w, av, grad_x=gxv)
        _check_backward(gy, total, mean, rstd, w, add, got)
        for i in range(6):
            assert (buf[i, :at] == 3.0).all() and (buf[i, at + size:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(10, 1), (9, 2), (11, 3), (6, 5), (5, 7), (8, 9)], ids=str)
def test_narrow_rows_between_nans(shape, fmt):
    """Rows narrower than 16 bytes, several of which end in the tensor's last 16:
    what follows and precedes the tensor is neither used nor written."""
    rows, width = shape
    x, w, b, gy, add = _inputs(rows, width, fmt, "f32", 11)
    size = x.numel()
    for shift in range(8):
        buf = torch.full((6, (size + 40) // 8 * 8), float("nan"), dtype=x.dtype, device=DEV)
        xv, gv, av, yv, tv, gxv = (buf[i, 8 + shift:8 + shift + size].view(x.shape) for i in range(6))
        xv.copy_(x), gv.copy_(gy), av.copy_(add)
        y, mean, rstd = wgs.layer_norm(xv, w, b, 1e-3, out=yv)
        _check_forward(x, w, b, 1e-3, y, mean, rstd)
        total, y, mean, rstd = wgs.residual_add_layer_norm(xv, av, w, b, 1e-3, residual_out=tv, out=yv)
        _check_forward(total, w, b, 1e-3, y, mean, rstd)
        got = wgs.layer_norm_bwd(gv, tv, mean, rstd, w, av, grad_x=gxv)
        _check_backward(gy, total, mean, rstd, w, add, got)
        for i in range(6):
            assert buf[i, :8 + shift].isnan().all() and buf[i, 8 + shift + size:].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("width", [96, 771, 1536])
def test_far_from_zero_outliers_and_constant_rows(width):
    x, w, b, gy, _ = _inputs(500, width, "f32", "f32", 11, offset=0.0)
    for far in (x + 1000.0, x - 30000.0):
        _check_forward(far, w, b, 1e-5, *wgs.layer_norm(far, w, b, 1e-5))
    out = x.clone()
    out[:, 0] = 5000.0
    _check_forward(out, w, b, 1e-5, *wgs.layer_norm(out, w, b, 1e-5))
    for value in (0.1, -60000.0, 0.0):
        flat = torch.full_like(x, value)
        y, mean, rstd = wgs.layer_norm(flat, w, b, 1e-5)
        # distances from the rounded mean are equal, and so is their mean but for
        # rounding: 2 (D + 3) u of a distance that is itself (D + 2) u of the value
        assert ((y - b).abs() <= 317 * w.abs() * (D + 3) ** 2 * 2 * U * U * abs(value) + U * b.abs()).all()
        assert (mean - value).abs().max() <= 2 * U * abs(value)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("width", [96, 771])
def test_bad_values_stay_in_their_row(bad, width):
    x, w, b, gy, _ = _inputs(300, width, "f16", "f32", 12)
    y, mean, rstd = wgs.layer_norm(x, w, b)
    want = (y, mean, rstd, wgs.layer_norm_bwd(gy, x, mean, rstd, w)[0])
    xb = x.clone()
    xb[77, 11] = bad
    y, mean, rstd = wgs.layer_norm(xb, w, b)
    gx = wgs.layer_norm_bwd(gy, xb, mean, rstd, w)[0]
    assert y[77].isnan().all() and mean[77].isnan() | mean[77].isinf() and rstd[77].isnan() and gx[77].isnan().all()
    for got, ref in zip((y, mean, rstd, gx), want):
        got[77] = ref[77]
        assert torch.equal(_bits(got), _bits(ref))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,width,fmt", [(131040, 192, "f16"), (32760, 1536, "bf16"), (32761, 771, "bf16"),
                                            (131040, 192, "f32"), (200000, 24, "bf16"), (3000, 8192, "f32")])
def test_large_calls(rows, width, fmt):
    x, w, b, gy, add = _inputs(rows, width, fmt, "f32", 13)
    total, y, mean, rstd = wgs.residual_add_layer_norm(x, add, w, b)
    assert torch.equal(_bits(total), _bits((x.float() + add.float()).to(x.dtype)))
    _check_forward(total, w, b, 1e-5, y, mean, rstd)
    got = wgs.layer_norm_bwd(gy, total, mean, rstd, w, add)
    _check_backward(gy, total, mean, rstd, w, add, got)
    assert _same(wgs.layer_norm_bwd(gy, total, mean, rstd, w, add), got)


@pytest.mark.gpu
def test_empty_calls_and_python_refusals():
    w, b = torch.ones(8, device=DEV), torch.zeros(8, device=DEV)
    x = torch.zeros(0, 8, device=DEV)
    y, mean, rstd = wgs.layer_norm(x, w, b)
    assert y.shape == (0, 8) and mean.shape == (0,)
    gx, gw, gb = wgs.layer_norm_bwd(x, x, mean, rstd, w, grad_weight=torch.ones_like(w))
    assert gx.shape == x.shape and (gw == 0).all() and (gb == 0).all()
    gx, gw, gb = wgs.layer_norm_bwd(x.half(), x.half(), mean, rstd, w.half(), grad_bias=w.half())
    assert (gw == 0).all() and (gb == 0).all()
    x = torch.randn(2, 4, 5, 8, device=DEV)
    y, mean, rstd = wgs.layer_norm(x, w, b)
    assert y.shape == x.shape and mean.shape == (2, 4, 5)
    flat = wgs.layer_norm(x.view(-1, 8), w, b)
    assert _same((y.view(-1, 8), mean.view(-1)), flat[:2])
    assert wgs.layer_norm(x[0, 0, 0], w, b)[1].shape == ()
    for args, kw in (((x, None, b), {}), ((x, w.half()), {}), ((x, w[:4]), {}), ((x, w, b[:4]), {}),
                     ((x.double(),), {}), ((x.transpose(1, 3),), {}), ((x, w, b), {"out": x.half()}),
                     ((x, w, b), {"mean": mean[:1]}), ((x.half(), w.bfloat16()), {}), ((x, 3), {}),
                     ((x, w, b.half()), {}), ((torch.zeros((), device=DEV),), {})):
        with pytest.raises(RuntimeError):
            wgs.layer_norm(*args, **kw)
    with pytest.raises(wgs.WgsError, match="WGS_ERR_WIDTH"):
        wgs.layer_norm(torch.zeros(2, 8193, device=DEV))
    with pytest.raises(RuntimeError, match="shape"):
        wgs.residual_add_layer_norm(x, x[:1])
    for kw in ({"weight": w, "workspace": torch.zeros(16, dtype=torch.uint8, device=DEV)}, {"grad_weight": w},
               {"grad_residual": x[:1]}, {"weight": w, "grad_x": x.half()}, {"weight": w, "grad_bias": w[:3]}):
        with pytest.raises(RuntimeError):
            wgs.layer_norm_bwd(x, x, mean, rstd, **kw)
    with pytest.raises(RuntimeError, match="shape"):
        wgs.layer_norm_bwd(x, x, mean[:1], rstd, w)


@pytest.mark.gpu
def test_statistics_and_parameter_gradients_may_be_left_out():
    """Through the C ABI: NULL statistics, and either gradient alone."""
    lib = _capi.load()
    rows, width = 700, 192
    x, w, b, gy, _ = _inputs(rows, width, "bf16", "f32", 3)
    want, mean, rstd = wgs.layer_norm(x, w, b)
    stream = torch.cuda.current_stream(DEV).cuda_stream
    y = torch.empty_like(x)
    assert lib.layer_norm(x.data_ptr(), w.data_ptr(), b.data_ptr(), y.data_ptr(), None, None, rows, width, 1e-5, 2,
                          0, stream) == OK
    assert _same((y,), (want,))
    full = wgs.layer_norm_bwd(gy, x, mean, rstd, w)
    ws = torch.empty(wgs.layer_norm_bwd_workspace_bytes(rows, width), dtype=torch.uint8, device=DEV)
    for keep in ((1, 0), (0, 1), (0, 0)):
        gx, gw, gb = torch.empty_like(x), torch.full_like(w, 7.0), torch.full_like(w, 7.0)
        any_kept = any(keep)
        assert lib.layer_norm_bwd(gy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), None,
                                  gx.data_ptr(), gw.data_ptr() if keep[0] else None,
                                  gb.data_ptr() if keep[1] else None, ws.data_ptr() if any_kept else None,
                                  ws.numel() if any_kept else 0, rows, width, 2, 0, stream) == OK
        assert _same((gx,), full[:1])
        assert _same((gw,), full[1:2]) if keep[0] else (gw == 7.0).all()
        assert _same((gb,), full[2:3]) if keep[1] else (gb == 7.0).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements in a call, checked in its first and last rows and
    in the columns' sums."""
    rows, width = 11_300_000, 192
    gen = torch.Generator(DEV).manual_seed(1)
    x = torch.empty(rows, width, dtype=torch.float16, device=DEV)
    gy = torch.empty_like(x)
    step = rows // 20
    for k in range(0, rows, step):
        x[k:k + step].normal_(generator=gen)
        gy[k:k + step].normal_(generator=gen)
    assert x.numel() > 2 ** 31
    w = torch.linspace(0.5, 1.5, width, device=DEV)
    y, mean, rstd = wgs.layer_norm(x, w, w)
    gx, gw, gb = wgs.layer_norm_bwd(gy, x, mean, rstd, w)
    for at in (slice(0, 100), slice(rows // 2, rows // 2 + 100), slice(rows - 100, rows)):
        _check_forward(x[at], w, w, 1e-5, y[at], mean[at], rstd[at])
        _check_backward(gy[at], x[at], mean[at], rstd[at], None, None,
                        (wgs.layer_norm_bwd(gy[at], x[at], mean[at], rstd[at])[0], None, None))
        assert torch.equal(gx[at], wgs.layer_norm_bwd(gy[at], x[at], mean[at], rstd[at], w)[0])
    want_w, want_b, mag_w, mag_b = (torch.zeros(width, dtype=torch.float64, device=DEV) for _ in range(4))
    for k in range(0, rows, step):
        h = (x[k:k + step].double() - mean[k:k + step, None].double()) * rstd[k:k + step, None].double()
        g = gy[k:k + step].double()
        want_w += (g * h).sum(0)
        mag_w += (g * h).abs().sum(0)
        want_b += g.sum(0)
        mag_b += g.abs().sum(0)
    for got, want, mag in ((gw, want_w, mag_w), (gb, want_b, mag_b)):
        assert ((got.double() - want).abs() <= (rows / 152 + 48) * U * mag).all()


# ---------------------------------------------------------- calls together ----

@pytest.mark.gpu
def test_graph_replay_and_streams_give_the_same_bits():
    """Captured calls replay next to eager ones on another stream, each with a
    workspace of its own."""
    x, w, b, gy, add = _inputs(900, 192, "bf16", "f32", 13)

    def run():
        t, y, mean, rstd = wgs.residual_add_layer_norm(x, add, w, b)
        return (t, y, mean, rstd, *wgs.layer_norm_bwd(gy, t, mean, rstd, w, add))

    want = run()
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            got = run()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(stream):
            graph.replay()
        eager = run()
        torch.cuda.synchronize()
        assert _same(got, want) and _same(eager, want)
        for t in got:
            t.zero_()


@pytest.mark.gpu
def test_calls_with_given_outputs_allocate_nothing():
    x, w, b, gy, add = _inputs(900, 192, "bf16", "f32", 3)
    t, y, gx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(900, device=DEV), torch.empty(900, device=DEV)
    gw, gb = torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(wgs.layer_norm_bwd_workspace_bytes(900, 192), dtype=torch.uint8, device=DEV)

    def calls():
        wgs.residual_add_layer_norm(x, add, w, b, residual_out=t, out=y, mean=mean, rstd=rstd)
        wgs.layer_norm_bwd(gy, t, mean, rstd, w, add, grad_x=gx, grad_weight=gw, grad_bias=gb, workspace=ws)

    calls()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    allocated, free = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0]
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == allocated
    assert torch.cuda.mem_get_info()[0] == free


@pytest.mark.gpu
def test_inputs_written_right_before_the_call():
    """Inputs written by the kernels just before, again and again with new
    values, with nothing between: no launch of a call may read what was there
    earlier."""
    for rows, width in ((30000, 192), (143, 90), (2000, 771), (500, 1536)):
        src = [_inputs(rows, width, "f16", "f32", k) for k in range(4)]
        own = [torch.zeros_like(t) for t in src[0]]
        x, w, b, gy, add = own

        def run(x, w, b, gy, add):
            t, y, mean, rstd = wgs.residual_add_layer_norm(x, add, w, b)
            return (t, y, mean, rstd, *wgs.layer_norm_bwd(gy, t, mean, rstd, w, add))

        got = []
        for _ in range(5):
            for given in src:
                for to, value in zip(own, given):
                    to.copy_(value)
                got.append(run(*own))
        torch.cuda.synchronize()
        for k, given in enumerate(src):
            want = run(*given)
            torch.cuda.synchronize()
            for r in range(5):
                assert _same(got[4 * r + k], want)


@pytest.mark.gpu
def test_two_streams_at_once():
    work = []
    for k, (rows, width, fmt) in enumerate(((5000, 96, "f32"), (3000, 771, "bf16"))):
        x, w, b, gy, add = _inputs(rows, width, fmt, "f32", k)

        def run(x=x, w=w, b=b, gy=gy, add=add):
            t, y, mean, rstd = wgs.residual_add_layer_norm(x, add, w, b)
            return (t, y, mean, rstd, *wgs.layer_norm_bwd(gy, t, mean, rstd, w, add))
        work.append(run)
    want = [run() for run in work]
    streams = [torch.cuda.Stream(DEV) for _ in work]
    torch.cuda.synchronize(DEV)
    for _ in range(3):
        got = []
        for run, stream in zip(work, streams):
            with torch.cuda.stream(stream):
                got.append([run() for _ in range(4)])
        torch.cuda.synchronize(DEV)
        for each, alone in zip(got, want):
            assert all(_same(outs, alone) for outs in each)
    wgs.check_error(DEV)
