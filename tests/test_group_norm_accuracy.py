"""Group norm's statistics where sums lose most, and its gradients over large
samples, against 64 bits with tolerances from the kernels' own depth.

With u = 2^-24, and D the additions on a value's way: a thread's rows, the row
groups of its block, a group's channels and the blocks' parts,

* mean: each sum is of distances from a reference, which a thread moves to its
  running mean after 8, 64, 512 ... rows.  A row that lies d from all others
  can leave the next 7n rows, after n, at d / n each: at most (8n)^2 / 2 roundings
  of u d / n, 32 n u d, in all no more than 37 u d times the thread's rows.  The
  group's distances from its mean come to about 2d with it, so
  |err| <= 20 D u mean|x - mean| + 2u |mean|.
* rstd: likewise the squares take 36 u d^2 before the first move and
  (8n)^2 / 2 (d / n)^2 u = 32 u d^2 after each, of which there are at most 5, where M2
  is at least d^2 - d^2 / rows.  With D u for the rest and D u for the joins of the
  blocks, var is off by (2D + 200) u and rstd by half: (D + 100) u + 8u.
* y, from the mean and rstd that the kernel gave: z = h w + b is off by
  3u (|h w| + |b|), an activation's slope is at most 1.13, and its own
  evaluation costs |y| (4u |t| + 16u), t the sigmoid's argument.
* the gradients, from the same: a slope is off by K = 5u max(|h w| + |b|) + 80u,
  so a sum by (D u + K + 4u) of its terms' magnitudes, and grad_x by
  (D u + K + 8u) of the magnitudes of its three.
* rounding to the output's format adds half a step.
"""
import math

import pytest
import torch

import window_gather_swin_gb300 as wgs

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

pytestmark = pytest.mark.gpu


def _depth(shape, fmt, backward):
    """D of a call: how many blocks share a sample, and a block's row
    groups, as the library chooses them from the sizes."""
    n, s, c, g = shape
    size = 4 if fmt == "f32" else 2
    chunks = c // (16 // size if c * size % 16 == 0 else 2 if c % 2 == 0 else 1)
    most, threads, parts = -(-s // 16), 512 if backward else 384, 1
    while parts < 8 and 2 * parts <= most and (n * parts < 608 or s * c >= 2 * parts * 65536):
        parts *= 2
    if s * c > 1 << 19 and n * parts < 304:
        parts = min(152 // n, most)
    elif n * parts > (100 if backward else 304):
        threads = 256
        want = -(-s // parts // 32) * chunks
        while n * parts > 304 and threads > 64 and threads // 2 >= want:
            threads //= 2
    groups = threads // min(chunks, threads)
    mine = -(-(-(-s // parts)) // groups)
    return mine + groups + c // g + parts + 32


def _slope(z, act):
    """act(z) and act'(z) in double."""
    if act is None:
        return z, torch.ones_like(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    k = 2 * math.sqrt(2 / math.pi)
    t = k * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(t)
    return z * s, s + z * s * torch.sigmoid(-t) * k * (1 + 3 * 0.044715 * z * z)


def _half(want, dtype):
    f = torch.finfo(dtype)
    return want.abs().clamp(min=f.smallest_normal) * (f.eps / 2)


def _check_statistics(x, mean, rstd, g, eps, D):
    n, s, c = x.shape
    for i in range(n):
        xd = x[i].double().view(s, g, c // g)
        m = xd.mean((0, 2))
        away = (xd - m[:, None]).abs()
        r = (away.square().mean((0, 2)) + eps).rsqrt()
        err = (mean[i].double() - m).abs() / (20 * D * U * away.mean((0, 2)) + 2 * U * m.abs())
        assert err.max() <= 1, ("mean", i, err.max().item())
        err = (rstd[i].double() / r - 1).abs() / ((D + 108) * U)
        assert err.max() <= 1, ("rstd", i, err.max().item())


def _check_output(x, y, w, b, mean, rstd, g, act):
    n, s, c = x.shape
    up = lambda v: v.double().repeat_interleave(c // g)
    for i in range(n):
        hw = (x[i].double() - up(mean[i])) * up(rstd[i]) * w.double()
        z = hw + b.double()
        want, _ = _slope(z, act)
        t = 1.6 * z.abs() + 0.0714 * z.abs() ** 3 if act == "gelu_tanh" else z.abs()
        tol = 1.13 * 3 * U * (hw.abs() + b.double().abs())
        if act is not None:
            tol = tol + want.abs() * (4 * U * t + 16 * U)
        err = (y[i].double() - want).abs() / (tol * (1 + torch.finfo(y.dtype).eps) + _half(want, y.dtype))
        assert err.max() <= 1, ("y", i, err.max().item())


def _weights(c, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    return (1 + 0.2 * torch.randn(c, generator=gen, device=DEV),
            0.2 * torch.randn(c, generator=gen, device=DEV))


# Short and long slabs, in two launches and in one by clusters.
OUTLIERS = [
    ((2, 3000, 32, 4), "f32"), ((1, 600_000, 16, 2), "f32"), ((4, 131040, 24, 4), "f32"),
    ((320, 16384, 16, 2), "f32"), ((1, 2_000_000, 8, 1), "f16"), ((6, 32760, 90, 6), "bf16"),
]


@pytest.mark.parametrize("where", ["first row", "eight rows", "last row"])
@pytest.mark.parametrize("shape,fmt", OUTLIERS, ids=str)
def test_statistics_beside_far_rows(shape, fmt, where):
    """Rows 5000 standard deviations from all others, where a sum starts and
    where it ends."""
    n, s, c, g = shape
    gen = torch.Generator(DEV).manual_seed(s)
    x = torch.randn(n, s, c, generator=gen, device=DEV) + torch.randn(c, generator=gen, device=DEV)
    rows = {"first row": slice(0, 1), "eight rows": slice(0, 8), "last row": slice(s - 1, s)}[where]
    x[:, rows] = 5000.0
    x = x.to(DT[fmt])
    w, b = _weights(c, 1)
    y, mean, rstd = wgs.group_norm_act(x, g, w, b, 1e-5, "silu")
    wgs.check_error(DEV)
    _check_statistics(x, mean, rstd, g, 1e-5, _depth(shape, fmt, False))
    _check_output(x, y, w, b, mean, rstd, g, "silu")


@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("shape,fmt", [((1, 131040, 192, 32), "f32"), ((1, 1_000_000, 8, 1), "f32"),
                                       ((2, 20000, 48, 4), "f32"), ((2, 4000, 1024, 1), "f16"),
                                       ((400, 300, 32, 4), "bf16")], ids=str)
def test_statistics_beside_a_far_slab(shape, fmt, where):
    """As many rows as a block takes, or an eighth of a sample where one cluster
    does, 100 deviations from all others: padding in front or behind."""
    n, s, c, g = shape
    gen = torch.Generator(DEV).manual_seed(s)
    x = 100 + torch.randn(n, s, c, generator=gen, device=DEV)
    rows = s // 8 if n * s < 200_000 else s * n // 152
    x[:, :rows] = 0
    x = (x if where == "first" else x.flip(1)).to(DT[fmt])
    w, b = _weights(c, 3)
    y, mean, rstd = wgs.group_norm_act(x, g, w, b, 1e-5, None)
    wgs.check_error(DEV)
    _check_statistics(x, mean, rstd, g, 1e-5, _depth(shape, fmt, False))
    _check_output(x, y, w, b, mean, rstd, g, None)


LARGE = [
    ((1, 131040, 192, 32), "f16", "silu"), ((3, 65600, 192, 32), "f16", "silu"),
    ((2, 131040, 192, 8), "bf16", "gelu_tanh"), ((33, 1000, 1001, 7), "bf16", "silu"),
    ((2, 20000, 770, 1), "f32", "gelu_tanh"), ((5, 32760, 384, 32), "bf16", None),
    ((3, 3000, 4096, 2048), "f32", "silu"), ((60, 700, 760, 95), "f16", "gelu_tanh"),
    ((400, 1000, 64, 8), "f32", "silu"), ((1, 40000, 99, 3), "f16", "gelu_tanh"),
]


@pytest.mark.parametrize("shape,fmt,act", LARGE, ids=str)
def test_large_samples_and_their_gradients(shape, fmt, act):
    """A gradient that is correlated with x and has a mean, so that the means
    over the groups and the weights' gradients are a large share of their
    terms: their absence would show, which is asserted too."""
    n, s, c, g = shape
    dtype = DT[fmt]
    gen = torch.Generator(DEV).manual_seed(c)
    noise = torch.randn(n, s, c, generator=gen, device=DEV)
    x = (noise * (0.5 + torch.rand(c, generator=gen, device=DEV))
         + torch.randn(c, generator=gen, device=DEV)).to(dtype)
    gy = (0.5 + 0.5 * noise + 0.5 * torch.randn(n, s, c, generator=gen, device=DEV)).to(dtype)
    del noise
    w, b = _weights(c, 2)
    y, mean, rstd = wgs.group_norm_act(x, g, w, b, 1e-5, act)
    gx, gw, gb = wgs.group_norm_act_bwd(gy, x, g, mean, rstd, w, b, act)
    wgs.check_error(DEV)
    _check_statistics(x, mean, rstd, g, 1e-5, _depth(shape, fmt, False))
    _check_output(x, y, w, b, mean, rstd, g, act)

    D = _depth(shape, fmt, True)
    up = lambda v: v.repeat_interleave(c // g)
    wd, bd = w.double(), b.double()
    want_w, want_b, mag_w, mag_b = (torch.zeros(c, dtype=torch.float64, device=DEV) for _ in range(4))
    zmax, rows = 0.0, []
    for i in range(n):
        r = rstd[i].double()
        h = (x[i].double() - up(mean[i].double())) * up(r)
        zmax = max(zmax, ((h * wd).abs().max() + bd.abs().max()).item())
        gyd = gy[i].double()
        dz = gyd * _slope(h * wd + bd, act)[1]
        want_w += (dz * h).sum(0)
        want_b += dz.sum(0)
        mag_w += (gyd * h).abs().sum(0)
        mag_b += gyd.abs().sum(0)
        d, size, hg = (v.view(s, g, -1) for v in (dz * wd, (gyd * wd).abs(), h))
        means = d.mean((0, 2))[:, None] + hg * (d * hg).mean((0, 2))[:, None]
        want = (r[:, None] * (d - means)).view(s, c)
        means = (r[:, None] * means).view(s, c)
        mag = (r[:, None] * (size + size.mean((0, 2))[:, None]
                             + hg.abs() * (size * hg.abs()).mean((0, 2))[:, None])).view(s, c)
        K = 5 * U * zmax + 80 * U
        tol = mag * (D * U + K + 8 * U) * (1 + torch.finfo(dtype).eps) + _half(want, dtype)
        err = (gx[i].double() - want).abs() / tol
        assert err.max() <= 1, ("grad_x", i, err.max().item())
        # a zero, or a grad_x without the group's means, would be outside
        rows.append(((want.abs() > 4 * tol).double().mean().item(),
                     (means.abs() > 4 * tol).double().mean().item()))
    assert min(min(v) for v in rows) > 0.5, rows
    K = 5 * U * zmax + 80 * U
    for got, want, mag in ((gw, want_w, mag_w), (gb, want_b, mag_b)):
        tol = mag * (D + n + K / U + 4) * U + U * want.abs()
        err = (got.double() - want).abs() / tol
        assert err.max() <= 1, err.max().item()
        assert (want.abs() > 4 * tol).double().mean() > 0.9
