"""Group norm with an activation over channels-last rows, and its gradients,
against the double-precision oracle.

Tolerances, with u = 2^-24 and D a bound on the additions that a value passes
through (the values of a group, at most 2048 on any path of the kernels):

* mean: |err| <= 2 D u S + 2u |mean|, S the largest |x - mean| of the group
  (the kernels sum distances from one of the values, at most 2 S).
* rstd: the squares summed are at most 4 S^2, so var is off by at most
  4 D u S^2 and rstd, relatively, by half of that over var + eps:
  R = 2 D u (S rstd)^2 + 8u.
* z = h w + b: |err| <= |w| rstd (err of the mean + u |x|) + |h w| (R + 4u)
  + 2u (|h w| + |b|); the activations' slopes are at most 1.13.
* the sigmoid's argument t (z, or the GELU's cubic) is off by 4u |t| from
  rounding and its exponential and reciprocal by 16u (hardware exp2 and
  reciprocal in 16-bit formats; less in FP32): |y| (4u |t| + 16u).
* gradients: given mean and rstd, h is off by 4u relatively and z by
  4u (|h w| + |b|); act' has slopes of at most 1.2 and its own evaluation
  errs by at most 64u (|t| <= 32, where it is not saturated), so dz is off by
  K |gy|, K = 5u max(|h w| + |b|) + 80u, and each output by (1.2 D u + K +
  8u) of the sum of its terms' magnitudes.
* rounding to the output's format adds half a step (half a subnormal step at
  the bottom).
"""
import math

import numpy as np
import pytest
import torch

import oracle
import window_gather_swin_gb300 as wgs
from window_gather_swin_gb300 import _capi

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OK, NULL, SHAPE, WIDTH, ALIGN, DTYPE, ARCH, LAUNCH, INDEX, ALIAS = range(10)
PTR = [0x10000000 * k for k in range(1, 14)]
NEED_FWD, NEED_BWD = "wgs_group_norm_act_workspace_bytes", "wgs_group_norm_act_bwd_workspace_bytes"


def _np(t, fmt):
    t = t.detach().cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if fmt == "bf16" else t.numpy()


def _values(t):
    return t.detach().cpu().double().numpy()


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def _half_step(want, dtype):
    f = torch.finfo(dtype)
    return np.maximum(np.abs(want), f.smallest_normal) * (f.eps / 2)


# ------------------------------------------------------------ the oracle ----

def _rand(shape, seed, std=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * std


@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
@pytest.mark.parametrize("n,s,c,g", [(2, 7, 12, 3), (1, 1, 6, 6), (3, 20, 5, 1)])
def test_oracle_equals_torch_in_double(n, s, c, g, act):
    x = _rand((n, s, c), 1).astype(np.float32)
    w, b = 1.0 + _rand(c, 2, 0.2), _rand(c, 3, 0.2)
    y, mean, rstd = oracle.group_norm_act(x, g, w, b, 1e-5, act, "f32")
    t = torch.from_numpy(x).double().permute(0, 2, 1)
    z = torch.nn.functional.group_norm(t, g, torch.from_numpy(w), torch.from_numpy(b), 1e-5) \
        if s * c // g > 1 else torch.from_numpy(b)[None, :, None].expand(n, c, s)
    want = {None: z, "silu": torch.nn.functional.silu(z),
            "gelu_tanh": torch.nn.functional.gelu(z, approximate="tanh")}[act]
    assert np.allclose(y, want.permute(0, 2, 1).numpy(), rtol=1e-12, atol=1e-12)
    flat = x.astype(np.float64).reshape(n, s, g, c // g)
    assert np.allclose(mean, flat.mean((1, 3)), rtol=1e-12, atol=1e-14)
    assert np.allclose(rstd, 1 / np.sqrt(flat.var((1, 3)) + 1e-5), rtol=1e-12)


@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
def test_oracle_gradient_equals_differences(act):
    """Central differences of sum(gy * y) in double: error O(step^2) + noise /
    step, both far below 1e-7 at a step of 1e-5 (values and slopes of order 1)."""
    n, s, c, g = 2, 5, 6, 2
    x, gy = _rand((n, s, c), 4).astype(np.float32), _rand((n, s, c), 5).astype(np.float32)
    w, b = 1.0 + _rand(c, 6, 0.2), _rand(c, 7, 0.2)
    _, mean, rstd = oracle.group_norm_act(x, g, w, b, 1e-3, act, "f32")
    (gx, gw, gb), _ = oracle.group_norm_act_bwd(gy, x, g, w, b, mean, rstd, act, "f32")

    def value(xd, wd, bd):
        f = xd.reshape(n, s, g, c // g)
        h = (f - f.mean((1, 3), keepdims=True)) / np.sqrt(f.var((1, 3), keepdims=True) + 1e-3)
        z = h.reshape(n, s, c) * wd + bd
        if act == "silu":
            z = z / (1 + np.exp(-z))
        elif act == "gelu_tanh":
            z = 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        return (z * gy.astype(np.float64)).sum()

    xd, h = x.astype(np.float64), 1e-5
    for which, grad in ((0, gx), (1, gw), (2, gb)):
        for i in np.ndindex(grad.shape):
            args = [xd.copy(), w.copy(), b.copy()]
            args[which][i] += h
            up = value(*args)
            args[which][i] -= 2 * h
            assert abs((up - value(*args)) / (2 * h) - grad[i]) < 1e-7


# --------------------------------------------------------------- refusals ----

def test_group_norm_refusals():
    """Every call here is refused while its arguments are checked."""
    lib = _capi.load()
    x, w, b, y, m, r, ws = PTR[:7]
    need = getattr(lib, NEED_FWD)(2, 100, 64, 8)

    def call(x=x, w=w, b=b, y=y, m=m, r=r, ws=ws, ws_bytes=need, n=2, spatial=100, channels=64,
             groups=8, act=1, dtype=1, param=0):
        return lib.group_norm_act(x, w, b, y, m, r, ws, ws_bytes, n, spatial, channels, groups, 1e-5,
                                  act, dtype, param, None)

    assert call(dtype=3) == DTYPE and call(param=2) == DTYPE and call(act=3) == DTYPE
    assert call(channels=4104, groups=8) == WIDTH and call(channels=4096, groups=4096) == WIDTH
    assert call(groups=7) == SHAPE and call(groups=0) == SHAPE and call(channels=0) == SHAPE
    assert call(n=-1) == SHAPE and call(spatial=-1) == SHAPE and call(n=65536) == SHAPE
    assert call(n=60000, spatial=2 ** 40) == SHAPE
    assert call(ws_bytes=need - 1) == SHAPE
    assert call(x=None, y=None, ws=None, n=0) == OK and call(x=None, spatial=0) == OK
    assert call(x=None) == NULL and call(y=None) == NULL and call(ws=None) == NULL
    assert call(w=None) == NULL and call(b=None) == NULL
    assert call(m=None) == NULL and call(r=None) == NULL
    assert call(x=x + 1) == ALIGN and call(y=y + 1) == ALIGN and call(ws=ws + 4) == ALIGN
    assert call(w=w + 2) == ALIGN and call(m=m + 2) == ALIGN
    assert call(y=x + 64) == ALIAS and call(y=w) == ALIAS and call(ws=x + 32) == ALIAS
    assert call(m=x + 32) == ALIAS and call(m=r) == ALIAS and call(r=ws + 16) == ALIAS
    assert call(ws=b) == ALIAS
    assert getattr(lib, NEED_FWD)(-1, 100, 64, 8) == 0 and getattr(lib, NEED_BWD)(2, 100, 64, 7) == 0


def test_group_norm_bwd_refusals():
    lib = _capi.load()
    gy, x, w, b, m, r, gx, gw, gb, ws = PTR[:10]
    need = getattr(lib, NEED_BWD)(2, 100, 64, 8)

    def call(gy=gy, x=x, w=w, b=b, m=m, r=r, gx=gx, gw=gw, gb=gb, ws=ws, ws_bytes=need, n=2,
             spatial=100, channels=64, groups=8, act=1, dtype=1, param=0):
        return lib.group_norm_act_bwd(gy, x, w, b, m, r, gx, gw, gb, ws, ws_bytes, n, spatial,
                                      channels, groups, act, dtype, param, None)

    assert call(dtype=-1) == DTYPE and call(param=2) == DTYPE and call(act=-1) == DTYPE
    assert call(channels=8192, groups=8) == WIDTH
    assert call(groups=7) == SHAPE and call(n=-1) == SHAPE and call(ws_bytes=need - 1) == SHAPE
    for name in ("gy", "x", "m", "r", "gx", "ws", "w", "b"):
        assert call(**{name: None}) == NULL, name
    assert call(w=None, b=None) == NULL                      # gradients of nothing
    assert call(gy=None, x=None, gx=None, gw=None, gb=None, ws=None, n=0) == OK
    assert call(gy=gy + 1) == ALIGN and call(gx=gx + 1) == ALIGN and call(ws=ws + 8) == ALIGN
    assert call(gw=gw + 2) == ALIGN and call(r=r + 1) == ALIGN
    assert call(gx=x + 64) == ALIAS and call(gx=gy + 64) == ALIAS and call(gw=w) == ALIAS
    assert call(gw=gb) == ALIAS and call(ws=x + 64) == ALIAS and call(gx=w) == ALIAS
    assert call(ws=m) == ALIAS and call(gb=r) == ALIAS


def test_python_refuses_cpu_tensors():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(RuntimeError, match="CUDA"):
        wgs.group_norm_act(x, 4)
    with pytest.raises(RuntimeError, match="CUDA"):
        wgs.group_norm_act_bwd(x, x, 4, torch.zeros(2, 4), torch.zeros(2, 4))
    assert wgs.group_norm_act_workspace_bytes(2, 100, 64, 8) > 0
    assert wgs.group_norm_act_bwd_workspace_bytes(2, 100, 64, 8) > 0


# -------------------------------------------------------------------- GPU ----

SHAPES = [  # n, spatial, channels, groups
    (1, 1, 1, 1), (1, 1, 64, 8), (2, 143, 90, 6), (1, 24, 192, 32), (3, 1000, 192, 32),
    (2, 577, 384, 32), (5, 33, 24, 24), (1, 4097, 8, 1), (2, 70, 1024, 16), (1, 50, 4096, 32),
    (2, 37, 2056, 8), (1, 300, 4095, 3), (9, 3, 40, 4), (1, 20011, 16, 2), (70, 65, 12, 3),
]
FORMATS = [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")]


def _inputs(shape, fmt, pfmt, seed, offset=1.0):
    n, s, c, g = shape
    gen = torch.Generator().manual_seed(seed)
    scale = 0.5 + torch.rand(c, generator=gen)
    x = (torch.randn(n, s, c, generator=gen) * scale + offset * torch.randn(c, generator=gen)).to(DT[fmt])
    w = (1 + 0.2 * torch.randn(c, generator=gen)).to(DT[pfmt])
    b = (0.2 * torch.randn(c, generator=gen)).to(DT[pfmt])
    gy = torch.randn(n, s, c, generator=gen).to(DT[fmt])
    return x, w, b, gy


def _t(z, act):
    z = np.abs(z)
    return 1.6 * z + 0.0714 * z ** 3 if act == "gelu_tanh" else z


def _spread(x, mean, g):
    n, s, c = x.shape
    return np.abs(x.reshape(n, s, g, c // g) - mean[:, None, :, None]).max((1, 3))


def _check_forward(x, w, b, g, eps, act, fmt, **kw):
    y, mean, rstd = wgs.group_norm_act(x, g, w, b, eps, act, **kw)
    n, s, c = x.shape
    xd = _values(x)
    wd = np.ones(c) if w is None else _values(w)
    bd = np.zeros(c) if b is None else _values(b)
    want, om, orr = oracle.group_norm_act(_np(x, fmt), g, wd, bd, np.float32(eps), act, fmt)
    z, _, _ = oracle.group_norm_act(_np(x, fmt), g, wd, bd, np.float32(eps), None, fmt)
    D = min(s * (c // g), 2048) + 8
    S = _spread(xd, om, g)
    tol_mean = 2 * D * U * S + 2 * U * np.abs(om)
    tol_r = 2 * D * U * (S * orr) ** 2 + 8 * U
    assert (np.abs(_values(mean) - om) <= tol_mean).all()
    assert (np.abs(_values(rstd) - orr) <= tol_r * orr).all()
    up = lambda v: np.repeat(v, c // g, 1)[:, None, :]
    hw = np.abs(z - bd)
    tz = np.abs(wd) * up(orr) * (up(tol_mean) + U * np.abs(xd)) + hw * (up(tol_r) + 4 * U) \
        + 2 * U * (hw + np.abs(bd))
    tol = 1.13 * tz + (0 if act in (None, "none") else np.abs(want) * (4 * U * _t(z, act) + 16 * U))
    tol = tol * (1 + torch.finfo(DT[fmt]).eps) + _half_step(want, DT[fmt])
    err = np.abs(_values(y) - want)
    assert (err <= tol).all(), (err / tol).max()
    return y, mean, rstd


def _check_backward(gy, x, w, b, g, mean, rstd, act, fmt, pfmt, **kw):
    gx, gw, gb = wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b, act, **kw)
    n, s, c = x.shape
    wd = np.ones(c) if w is None else _values(w)
    bd = np.zeros(c) if b is None else _values(b)
    want, mag = oracle.group_norm_act_bwd(_np(gy, fmt), _np(x, fmt), g, wd, bd, _values(mean),
                                          _values(rstd), act, fmt)
    h = (_values(x).reshape(n, s, g, -1) - _values(mean)[:, None, :, None]) * _values(rstd)[:, None, :, None]
    z = np.abs(h.reshape(n, s, c) * wd).max() + np.abs(bd).max()
    D = min(n * s * (c // g), 2048) + 8
    K = 5 * U * z + 80 * U
    for got, ref, m, f in ((gx, want[0], mag[0], fmt), (gw, want[1], mag[1], pfmt), (gb, want[2], mag[2], pfmt)):
        if got is None:
            assert w is None
            continue
        tol = m * (1.2 * D * U + K + 8 * U) * (1 + torch.finfo(DT[f]).eps) + _half_step(ref, DT[f])
        err = np.abs(_values(got) - ref)
        assert got.shape == ref.shape and (err <= tol).all(), (err / tol).max()
    return gx, gw, gb


@pytest.mark.gpu
@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
@pytest.mark.parametrize("fmt,pfmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_group_norm_and_gradients(shape, fmt, pfmt, act):
    x, w, b, gy = (t.to(DEV) for t in _inputs(shape, fmt, pfmt, sum(shape)))
    n, s, c, g = shape
    need = wgs.group_norm_act_workspace_bytes(n, s, c, g)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)    # NaN patterns
    y, mean, rstd = _check_forward(x, w, b, g, 1e-5, act, fmt, workspace=ws)
    assert (ws[need:] == 0xff).all()
    need = wgs.group_norm_act_bwd_workspace_bytes(n, s, c, g)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)
    gx, gw, gb = _check_backward(gy, x, w, b, g, mean, rstd, act, fmt, pfmt, workspace=ws)
    assert (ws[need:] == 0xff).all()
    # a fixed order of additions; in place gives the same
    y2, m2, r2 = wgs.group_norm_act(x.clone(), g, w, b, 1e-5, act)
    assert torch.equal(_bits(y), _bits(y2)) and torch.equal(mean, m2) and torch.equal(rstd, r2)
    inplace = x.clone()
    wgs.group_norm_act(inplace, g, w, b, 1e-5, act, out=inplace)
    assert torch.equal(_bits(inplace), _bits(y))
    for over in (0, 1):
        gyc, xc = gy.clone(), x.clone()
        got = wgs.group_norm_act_bwd(gyc, xc, g, mean, rstd, w, b, act, grad_x=(gyc, xc)[over])
        assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(got, (gx, gw, gb)))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_group_norm_without_weights_on_unaligned_views(fmt):
    shape = (2, 57, 64, 4)
    n, s, c, g = shape
    x, w, b, gy = _inputs(shape, fmt, "f32", 9)
    size = x.numel()
    buf = torch.full((3, size + 16), 3.0, dtype=x.dtype, device=DEV)
    xv, gv, yv = (buf[i, 1:1 + size].view(x.shape) for i in range(3))
    xv.copy_(x)
    gv.copy_(gy)
    y, mean, rstd = _check_forward(xv, None, None, g, 1e-3, "silu", fmt, out=yv)
    gx, gw, gb = _check_backward(gv, xv, None, None, g, mean, rstd, "silu", fmt, "f32", grad_x=yv)
    assert gw is None and gb is None
    assert (buf[:, 0] == 3.0).all() and (buf[:, 1 + size:] == 3.0).all()


@pytest.mark.gpu
def test_group_norm_far_from_zero_and_outliers():
    """A mean 1000 standard deviations away, one value far from all others in
    the first place that a sum could start from, and constant groups."""
    shape = (2, 3000, 32, 4)
    x, w, b, gy = (t.to(DEV) for t in _inputs(shape, "f32", "f32", 11, offset=0.0))
    far = x + 1000.0
    _check_forward(far, w, b, 4, 1e-5, None, "f32")
    out = x.clone()
    out[:, 0, :] = 5000.0
    _check_forward(out, w, b, 4, 1e-5, "silu", "f32")
    flat = torch.full_like(x, 0.1)
    y, mean, rstd = wgs.group_norm_act(flat, 4, w, b, 1e-5, None)
    assert torch.equal(mean, torch.full_like(mean, np.float32(0.1)))
    assert torch.equal(y, b.expand_as(y).contiguous())
    z, _, _ = wgs.group_norm_act(torch.full_like(x, 60000.0).half(), 4, w.half(), b.half(), 1e-5, None)
    assert torch.equal(z, b.half().expand_as(z).contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_group_norm_keeps_bad_values_in_their_group(bad):
    shape = (2, 200, 32, 4)
    x, w, b, gy = (t.to(DEV) for t in _inputs(shape, "f16", "f32", 12))
    want = wgs.group_norm_act(x, 4, w, b, 1e-5, "silu")[0]
    x[1, 77, 11] = bad
    y = wgs.group_norm_act(x, 4, w, b, 1e-5, "silu")[0]
    assert y[1, :, 8:16].isnan().all()
    y[1, :, 8:16] = want[1, :, 8:16]
    assert torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activations_far_out(act):
    """z far from zero: the activation is z or 0 and its slope 1 or 0, with
    nothing that overflows on the way (two values -1 and 1 have mean 0 and
    variance 1 exactly, and the weight takes z out)."""
    x = torch.tensor([-1.0, 1.0], device=DEV).view(1, 2, 1)
    for w in (128.0, 2.0 ** 20, 2.0 ** 50, 2.0 ** 100):
        wt, bt = torch.tensor([w], device=DEV), torch.zeros(1, device=DEV)
        y, mean, rstd = wgs.group_norm_act(x, 1, wt, bt, 0.0, act)
        assert mean.item() == 0.0 and rstd.item() == 1.0
        assert y[0, 1, 0].item() == w and abs(y[0, 0, 0].item()) <= 1e-30
        gx, gw, gb = wgs.group_norm_act_bwd(torch.ones_like(x), x, 1, mean, rstd, wt, bt, act)
        assert gx.isfinite().all() and gw.item() == 1.0 and gb.item() == 1.0


@pytest.mark.gpu
def test_group_norm_empty_and_python_refusals():
    w, b = torch.ones(8, device=DEV), torch.zeros(8, device=DEV)
    for shape in ((0, 5, 8), (3, 0, 8)):
        x = torch.zeros(shape, device=DEV)
        y, mean, rstd = wgs.group_norm_act(x, 2, w, b)
        assert y.shape == x.shape and mean.shape == (shape[0], 2)
        gx, gw, gb = wgs.group_norm_act_bwd(x, x, 2, mean, rstd, w, b)
        assert gx.shape == x.shape and (gw == 0).all() and (gb == 0).all()
    x = torch.zeros(2, 4, 4, 8, device=DEV)
    y, mean, rstd = wgs.group_norm_act(x, 2, w, b)
    assert y.shape == x.shape
    for args, kw in (((x, 3), {}), ((x, 0), {}), ((x, 2, w), {}), ((x, 2, w, b.half()), {}),
                     ((x, 2, w[:4], b[:4]), {}), ((x, 2, w, b), {"act": "relu"}),
                     ((x.double(), 2), {}), ((x.transpose(1, 3), 2), {}),
                     ((x, 2, w, b), {"out": x.half()}), ((x, 2, w, b), {"mean": mean.t()}),
                     ((x, 2, w, b), {"workspace": x}), ((x.half(), 2, w.bfloat16(), b.bfloat16()), {})):
        with pytest.raises(RuntimeError):
            wgs.group_norm_act(*args, **kw)
    with pytest.raises(wgs.WgsError, match="WGS_ERR_WIDTH"):
        wgs.group_norm_act(torch.zeros(1, 2, 4104, device=DEV), 8)
    with pytest.raises(wgs.WgsError, match="WGS_ERR_SHAPE"):
        wgs.group_norm_act(x, 2, w, b, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    for kw in ({"weight": w}, {"grad_weight": w}, {"weight": w, "bias": b, "grad_x": x.half()}):
        with pytest.raises(RuntimeError):
            wgs.group_norm_act_bwd(x, x, 2, mean, rstd, **kw)
    with pytest.raises(RuntimeError, match="shape"):
        wgs.group_norm_act_bwd(x, x, 2, mean[:1], rstd, w, b)


@pytest.mark.gpu
def test_graph_replay_and_streams_give_the_same_bits():
    """Captured calls replay next to eager ones on another stream, each with a
    workspace of its own."""
    shape = (3, 900, 192, 32)
    n, s, c, g = shape
    x, w, b, gy = (t.to(DEV) for t in _inputs(shape, "bf16", "f32", 13))
    y, mean, rstd = wgs.group_norm_act(x, g, w, b)
    want = (y,) + wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            y1, m1, r1 = wgs.group_norm_act(x, g, w, b)
            got = (y1,) + wgs.group_norm_act_bwd(gy, x, g, m1, r1, w, b)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(stream):
            graph.replay()
        y2, m2, r2 = wgs.group_norm_act(x, g, w, b)
        eager = (y2,) + wgs.group_norm_act_bwd(gy, x, g, m2, r2, w, b)
        torch.cuda.synchronize()
        for p, q, r in zip(want, got, eager):
            assert torch.equal(_bits(p), _bits(q)) and torch.equal(_bits(p), _bits(r))
        for t in got:
            t.zero_()


# The launches for samples that one cluster does not hold: one batch (two
# launches), and several batches (a launch whose blocks take them in turn),
# with whole and odd rows.
LARGE = [
    ((1, 131040, 192, 32), "f16", "silu"), ((3, 65600, 192, 32), "f16", "silu"),
    ((2, 131040, 192, 8), "bf16", "gelu_tanh"), ((33, 1000, 1001, 7), "bf16", "silu"),
    ((2, 20000, 770, 1), "f32", "gelu_tanh"), ((5, 32760, 384, 32), "bf16", None),
    ((3, 3000, 4096, 2048), "f32", "silu"), ((60, 700, 760, 95), "f16", "gelu_tanh"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape,fmt,act", LARGE, ids=str)
def test_large_samples(shape, fmt, act):
    """As above, against the formulas in double precision on the GPU."""
    n, s, c, g = shape
    dtype = DT[fmt]
    x, w, b, gy = (t.to(DEV) for t in _inputs((1, s, c, g), fmt, "f32", c))
    gen = torch.Generator(DEV).manual_seed(5)
    x, gy = ((torch.randn(n, s, c, generator=gen, device=DEV) * (1 + t[0, :1].float().abs())).to(dtype)
             for t in (x, gy))
    y, mean, rstd = wgs.group_norm_act(x, g, w, b, 1e-5, act)
    gx, gw, gb = wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b, act)
    wgs.check_error(DEV)
    D, half = 2056, torch.finfo(dtype).eps / 2
    want_gw, want_gb, mag_w, mag_b = (torch.zeros(c, dtype=torch.float64, device=DEV) for _ in range(4))
    K = 0.0
    for i in range(n):
        xd = x[i].double().view(s, g, c // g)
        m, var = xd.mean((0, 2)), xd.var((0, 2), unbiased=False)
        r = (var + 1e-5).rsqrt()
        S = (xd - m[:, None]).abs().amax((0, 2))
        tol_m, tol_r = 2 * D * U * S + 2 * U * m.abs(), 2 * D * U * (S * r) ** 2 + 8 * U
        assert ((mean[i].double() - m).abs() <= tol_m).all()
        assert ((rstd[i].double() - r).abs() <= tol_r * r).all()
        up = lambda v: v.repeat_interleave(c // g)
        wd, bd = w.double(), b.double()
        h = ((xd - m[:, None]) * r[:, None]).view(s, c)
        z = (h * wd + bd).requires_grad_()
        ref = {None: lambda v: v * 1.0, "silu": torch.nn.functional.silu,
               "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](z)
        ref.sum().backward()
        slope, ref, z, hw = z.grad, ref.detach(), z.detach(), (h * wd).abs()
        t = 1.6 * z.abs() + 0.0714 * z.abs() ** 3 if act == "gelu_tanh" else z.abs()
        tz = wd.abs() * up(r) * (up(tol_m) + U * x[i].double().abs()) + hw * (up(tol_r) + 4 * U) \
            + 2 * U * (hw + bd.abs())
        tol = (1.13 * tz + ref.abs() * (4 * U * t + 16 * U)) * (1 + half * 2) + half * ref.abs() + 1e-7 * half
        err = (y[i].double() - ref).abs()
        assert (err <= tol).all(), (err / tol).max()
        # the gradients, from the statistics that the forward gave
        m, r = mean[i].double(), rstd[i].double()
        h = ((xd - m[:, None]) * r[:, None]).view(s, c)
        K = max(K, 5 * U * (hw.max() + bd.abs().max()).item() + 80 * U)
        gyd = gy[i].double()
        dz = gyd * slope          # the slope moves by less than the bound below with the statistics
        d, size = (dz * wd).view(s, g, -1), (gyd * wd).abs().view(s, g, -1)
        hg = h.view(s, g, -1)
        want = (r[:, None] * (d - d.mean((0, 2))[:, None] - hg * (d * hg).mean((0, 2))[:, None])).view(s, c)
        mag = (r[:, None] * (size + size.mean((0, 2))[:, None]
                             + hg.abs() * (size * hg.abs()).mean((0, 2))[:, None])).view(s, c)
        slack = 1.2 * D * U + K + 8 * U + 1.2 * tz.max().item()
        err = (gx[i].double() - want).abs()
        assert (err <= mag * slack * 1.01 + half * want.abs() + 1e-7 * half).all(), (err / mag).max()
        want_gw += (dz * h).sum(0)
        want_gb += dz.sum(0)
        mag_w += (gyd * h).abs().sum(0)
        mag_b += gyd.abs().sum(0)
    for got, want, mag in ((gw, want_gw, mag_w), (gb, want_gb, mag_b)):
        assert ((got.double() - want).abs() <= mag * slack + U * want.abs()).all()
    # the same call again, and in place, gives the same bits
    y2, mean2, _ = wgs.group_norm_act(x.clone(), g, w, b, 1e-5, act)
    again = wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b, act, grad_x=gy)
    assert torch.equal(_bits(y2), _bits(y)) and torch.equal(mean2, mean)
    assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(again, (gx, gw, gb)))
    wgs.group_norm_act(x, g, w, b, 1e-5, act, out=x)
    assert torch.equal(_bits(x), _bits(y))


# Samples that are many enough to fill the GPU: fewer blocks a sample and fewer
# threads a block, more samples than blocks that are resident, one position each.
MANY = [(1300, 49, 24, 3), (700, 20, 40, 8), (313, 70, 136, 17), (5000, 1, 64, 8), (2500, 3, 15, 5),
        (90, 130, 64, 32), (13, 520, 90, 45)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,pfmt", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_many_samples(shape, fmt, pfmt):
    g = shape[3]
    act = "gelu_tanh" if fmt == "f16" else "silu"
    x, w, b, gy = (t.to(DEV) for t in _inputs(shape, fmt, pfmt, 11))
    y, mean, rstd = _check_forward(x, w, b, g, 1e-5, act, fmt)
    first = _check_backward(gy, x, w, b, g, mean, rstd, act, fmt, pfmt)
    again = wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b, act)
    assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(first, again))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements in a call, checked in the last sample's first and
    last groups and in its first and last rows."""
    n, s, c, g = 2, 5_700_000, 192, 32
    gen = torch.Generator(DEV).manual_seed(1)
    x = torch.empty(n, s, c, dtype=torch.float16, device=DEV)
    gy = torch.empty_like(x)
    for i in range(n):
        x[i].normal_(generator=gen)
        gy[i].normal_(generator=gen)
    assert x.numel() > 2 ** 31
    w = torch.linspace(0.5, 1.5, c, device=DEV)
    b = torch.linspace(-0.2, 0.2, c, device=DEV)
    y, mean, rstd = wgs.group_norm_act(x, g, w, b, 1e-5, "silu")
    gx, gw, gb = wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b, "silu")
    D, half = 2 ** 17, 2.0 ** -11      # a slab's 37500 rows of 6 channels, and the joins
    for i, j in ((0, 0), (n - 1, 0), (n - 1, g - 1)):
        at = slice(j * c // g, (j + 1) * c // g)
        xd, gd = x[i, :, at].double(), gy[i, :, at].double()
        m, r = xd.mean(), (xd.var(unbiased=False) + 1e-5).rsqrt()
        S = (xd - m).abs().max()
        assert (mean[i, j] - m).abs() <= 2 * D * U * S
        assert (rstd[i, j] / r - 1).abs() <= 2 * D * U * (S * r) ** 2
        m, r = mean[i, j].double(), rstd[i, j].double()
        h = (xd - m) * r
        z = h * w[at].double() + b[at].double()
        sig = torch.sigmoid(z)
        assert ((y[i, :, at].double() - z * sig).abs() <= half * (z * sig).abs() + 2e-6).all()
        d = gd * (sig + z * sig * (1 - sig)) * w[at].double()
        want = r * (d - d.mean() - h * (d * h).mean())
        assert ((gx[i, :, at].double() - want).abs() <= half * want.abs() + 5e-6 * gd.abs() + 1e-5).all()
    gwant = torch.zeros(c, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(gwant)
    for i in range(n):
        for k in range(0, s, s // 20):
            rows = slice(k, min(s, k + s // 20))
            up = lambda v: v[i].double().repeat_interleave(c // g)
            h = (x[i, rows].double() - up(mean)) * up(rstd)
            z = h * w.double() + b.double()
            sig = torch.sigmoid(z)
            dz = gy[i, rows].double() * (sig + z * sig * (1 - sig))
            gwant += dz.sum(0)
            mag += dz.abs().sum(0)
    assert ((gb.double() - gwant).abs() <= 40000 * U * mag).all()


@pytest.mark.gpu
def test_calls_with_given_outputs_allocate_nothing():
    n, s, c, g = 3, 900, 192, 32
    x, w, b, gy = (t.to(DEV) for t in _inputs((n, s, c, g), "bf16", "f32", 3))
    y, gx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(n, g, device=DEV), torch.empty(n, g, device=DEV)
    gw, gb = torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(wgs.group_norm_act_bwd_workspace_bytes(n, s, c, g), dtype=torch.uint8, device=DEV)
    assert ws.numel() >= wgs.group_norm_act_workspace_bytes(n, s, c, g)

    def calls():
        wgs.group_norm_act(x, g, w, b, out=y, mean=mean, rstd=rstd, workspace=ws)
        wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b, grad_x=gx, grad_weight=gw, grad_bias=gb,
                               workspace=ws)

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
    """x, the weights and grad_y written by the kernels just before, again and
    again with new values, with nothing between: no launch of a call may read
    what was there earlier."""
    for n, s, c, g in ((1, 30000, 192, 32), (2, 143, 90, 6)):
        x = torch.zeros(n, s, c, dtype=torch.float16, device=DEV)
        gy, w, b = torch.zeros_like(x), torch.zeros(c, device=DEV), torch.zeros(c, device=DEV)
        src = [[t.to(DEV) for t in _inputs((n, s, c, g), "f16", "f32", k)] for k in range(4)]
        got = []
        for _ in range(5):
            for sx, sw, sb, sg in src:
                x.copy_(sx)
                gy.copy_(sg)
                w.copy_(sw)
                b.copy_(sb)
                y, mean, rstd = wgs.group_norm_act(x, g, w, b)
                got.append((y,) + wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b))
        torch.cuda.synchronize()
        for k, (sx, sw, sb, sg) in enumerate(src):
            y, mean, rstd = wgs.group_norm_act(sx, g, sw, sb)
            torch.cuda.synchronize()
            want = (y,) + wgs.group_norm_act_bwd(sg, sx, g, mean, rstd, sw, sb)
            for r in range(5):
                assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(got[4 * r + k], want))
