"""A run of the embedding and layer-norm operators as a block uses them: tokens
looked up in a table, a branch joined to the residual stream and normalised with
weight and bias, a hidden layer with the bias + GELU epilogue, and the way back to
the gradients of the table, the norm's weights and the hidden layer's bias.  The
dense products are torch's, in the tokens' 16-bit format; the yardstick is torch
autograd in float64 on the same values.

Tolerance: the path rounds to 16 bits at 13 places (lookup, branch, their sum, norm,
hidden product, bias, GELU; on the way back the GELU's, both products', the norm's
and the branch's gradients, their sum, and a gradient's own rounding), each at most
eps / 2 of its tensor; a factor of two covers what the norm and the GELU amplify.
Measured as the norm of the error over the norm of the gradient: 26 * eps / 2.
"""
import math

import pytest
import torch

import window_gather_swin_gb300 as wgs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5


def _problem(n, rows, width, hidden, dtype):
    g = torch.Generator().manual_seed(31)
    rand = lambda *s: torch.randn(*s, generator=g)
    p = {"table": 0.5 * rand(rows, width), "proj": rand(width, width) / math.sqrt(width),
         "w": 1 + 0.2 * rand(width), "b": 0.2 * rand(width), "up": rand(width, hidden) / math.sqrt(width),
         "b1": 0.2 * rand(hidden), "grad": rand(n, hidden), "grad_r": rand(n, width)}
    p = {k: v.to(dtype).to(DEV) for k, v in p.items()}
    idx = (rows * torch.rand(n, generator=g) ** 2).int()
    idx[::17] = -1
    p["idx"] = idx.to(DEV)
    return p


def _library(p, scale):
    dtype, rows = p["up"].dtype, p["table"].shape[0]
    x = wgs.embedding(p["table"], p["idx"], scale)
    r, y, mean, rstd = wgs.residual_add_layer_norm(x, x @ p["proj"], p["w"], p["b"], EPS)
    h = y @ p["up"]
    out = wgs.bias_gelu_tanh(h, p["b1"])
    gh, gb1 = wgs.bias_gelu_tanh_bwd(p["grad"], h, p["b1"])
    gr, gw, gb = wgs.layer_norm_bwd(gh @ p["up"].t(), r, mean, rstd, p["w"], p["grad_r"])
    gx = gr + gr @ p["proj"].t()
    gt = wgs.embedding_bwd(gx, p["idx"], rows, scale, dtype)
    wgs.check_error(DEV)
    return out, gt, gw, gb, gb1


def _autograd(p, scale):
    d = {k: v.double().requires_grad_() if v.is_floating_point() else v for k, v in p.items()}
    idx = p["idx"].long()
    x = torch.where((idx >= 0)[:, None], d["table"][idx.clamp(min=0)] * scale, 0.0)
    r = x + x @ d["proj"]
    y = torch.nn.functional.layer_norm(r, r.shape[-1:], d["w"], d["b"], EPS)
    out = torch.nn.functional.gelu(y @ d["up"] + d["b1"], approximate="tanh")
    ((out * d["grad"].detach()).sum() + (r * d["grad_r"].detach()).sum()).backward()
    return out.detach(), d["table"].grad, d["w"].grad, d["b"].grad, d["b1"].grad


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", [(700, 50, 192, 768), (5000, 366, 96, 384), (3001, 2000, 104, 200)], ids=str)
def test_block_gradients(shape, dtype):
    p, scale = _problem(*shape, dtype), 1.5
    bound = 26 * torch.finfo(dtype).eps / 2
    for name, got, want in zip(("out", "table", "w", "b", "b1"), _library(p, scale), _autograd(p, scale)):
        err = (got.double() - want).norm() / want.norm()
        assert err < bound, (name, err.item(), bound)


def test_calls_on_two_streams_at_once():
    """Runs that overlap on the GPU, each with its own inputs, give the bits that
    they give alone."""
    work = [(_problem(4000, 100 * (k + 1), 192, 384, torch.bfloat16), 1.0 + k) for k in range(2)]

    def run(p, scale):
        x = wgs.embedding(p["table"], p["idx"], scale)
        r, y, mean, rstd = wgs.residual_add_layer_norm(x, x, p["w"], p["b"], EPS)
        gr, gw, gb = wgs.layer_norm_bwd(y, r, mean, rstd, p["w"], p["grad_r"])
        return x, r, y, gr, gw, gb, wgs.embedding_bwd(gr, p["idx"], p["table"].shape[0], scale)

    want = [run(*w) for w in work]
    streams = [torch.cuda.Stream(DEV) for _ in work]
    torch.cuda.synchronize(DEV)
    for _ in range(3):
        got = []
        for w, stream in zip(work, streams):
            with torch.cuda.stream(stream):
                got.append([run(*w) for _ in range(4)])
        torch.cuda.synchronize(DEV)
        for each, alone in zip(got, want):
            for outs in each:
                assert all(torch.equal(a, b) for a, b in zip(outs, alone))
