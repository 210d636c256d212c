"""A run of the training operators as a shifted-window block uses them: group
norm + SiLU on the token grid, window gather, attention with a learned
position bias per latitude band and the shift mask, window reverse, and the
way back to the gradients of the tokens, the norm's weights and the bias
table.  The dense products are torch's, in the tokens' 16-bit format; the
yardstick is torch autograd in float64 on the same values.

Tolerance: the path rounds to 16 bits at about 16 places (norm output, qkv,
logits twice, probabilities, their products and the same on the way back),
each at most eps / 2 of its tensor; a factor of two covers the softmax's and
the norm's amplification.  Measured as the norm of the error over the norm
of the gradient: 32 * eps / 2.
"""
import math

import pytest
import torch

import window_gather_swin_gb300 as wgs
from window_gather_swin_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
HEADS, GROUPS, C = 6, 32, 192
N = synth.WINDOW[0] * synth.WINDOW[1] * synth.WINDOW[2]


def _problem(stage, dtype):
    g = torch.Generator().manual_seed(21)
    p = {
        "x": torch.randn(stage.tokens, C, generator=g) + torch.randn(C, generator=g),
        "w": 1 + 0.2 * torch.randn(C, generator=g),
        "b": 0.2 * torch.randn(C, generator=g),
        "qkv": torch.randn(C, 3 * C, generator=g) / math.sqrt(C),
        "grad": torch.randn(stage.tokens, C, generator=g),
    }
    p = {k: v.to(dtype).to(DEV) for k, v in p.items()}
    bands = stage.windowed_rows // N // (stage.padded[2] // synth.WINDOW[2])
    buckets = wgs.window_bucket_count(synth.WINDOW, 3)
    p["table"] = (0.5 * torch.randn(bands, buckets, HEADS, generator=g)).to(DEV)
    p["type"] = (torch.arange(stage.windowed_rows // N) // (stage.padded[2] // synth.WINDOW[2])).int().to(DEV)
    return p


def _maps(stage):
    m = {k: f(stage.grid, synth.WINDOW, synth.SHIFT, device=DEV)
         for k, f in (("idx", wgs.build_window_index), ("inv", wgs.build_window_inverse),
                      ("region", wgs.build_shift_regions))}
    m["bucket"] = wgs.build_window_buckets(synth.WINDOW, 3)
    return m


def _library(p, m):
    dtype = p["x"].dtype
    bands, buckets, _ = p["table"].shape
    plan = wgs.build_bucket_plan(m["bucket"], buckets, device=DEV)
    x = p["x"][None]
    y, mean, rstd = wgs.group_norm_act(x, GROUPS, p["w"], p["b"], EPS, "silu")
    win = wgs.window_gather(y[0], m["idx"])
    qkv = (win @ p["qkv"]).view(-1, N, 3, HEADS, C // HEADS).permute(2, 0, 3, 1, 4)
    q, k, v = qkv[0], qkv[1], qkv[2]
    scale = (C // HEADS) ** -0.5
    bias = wgs.position_bias(p["table"], m["bucket"].to(DEV), dtype=dtype)
    logits = wgs.window_bias_mask_add(((q @ k.transpose(-1, -2)) * scale).contiguous(), bias, p["type"],
                                      m["region"], -100.0)
    prob = torch.softmax(logits.float(), -1)
    # the way back, from the gradient of the block's tokens
    go = wgs.window_gather(p["grad"], m["idx"]).view(-1, N, HEADS, C // HEADS).transpose(1, 2)
    gp = (go @ v.transpose(-1, -2)).float()
    gs = (prob * (gp - (prob * gp).sum(-1, keepdim=True))).to(dtype)
    g_table = wgs.position_bias_bwd(gs, plan, p["type"], bands)
    gq, gk = gs @ k * scale, gs.transpose(-1, -2) @ q * scale
    gv = prob.to(dtype).transpose(-1, -2) @ go
    gwin = torch.stack([gq, gk, gv]).permute(1, 3, 0, 2, 4).reshape(-1, 3 * C) @ p["qkv"].t()
    gy = wgs.window_gather(gwin, m["inv"])
    gx, gw, gb = wgs.group_norm_act_bwd(gy[None], x, GROUPS, mean, rstd, p["w"], p["b"], "silu")
    wgs.check_error(DEV)
    return gx[0], gw, gb, g_table


def _autograd(p, m):
    d = {k: v.double().requires_grad_() if v.is_floating_point() else v for k, v in p.items()}
    z = torch.nn.functional.group_norm(d["x"].t()[None], GROUPS, d["w"], d["b"], EPS)[0].t()
    y = torch.nn.functional.silu(z)
    idx = m["idx"].long()
    win = torch.where((idx >= 0)[:, None], y[idx.clamp(min=0)], 0.0)
    qkv = (win @ d["qkv"]).view(-1, N, 3, HEADS, C // HEADS).permute(2, 0, 3, 1, 4)
    bias = d["table"][:, m["bucket"].to(DEV).long()].permute(0, 3, 1, 2)[d["type"].long()]
    lab = m["region"].view(-1, N)
    mask = torch.where(lab[:, :, None] == lab[:, None, :], 0.0, -100.0)[:, None]
    s = qkv[0] @ qkv[1].transpose(-1, -2) * (C // HEADS) ** -0.5 + bias + mask
    o = (torch.softmax(s, -1) @ qkv[2]).transpose(1, 2).reshape(-1, C)[m["inv"].long()]
    (o * d["grad"].detach()).sum().backward()
    return d["x"].grad, d["w"].grad, d["b"].grad, d["table"].grad


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("stage", [synth.TINY, synth.TINY_PADDED], ids=lambda s: s.name)
def test_block_gradients(stage, dtype):
    p, m = _problem(stage, dtype), _maps(stage)
    bound = 32 * torch.finfo(dtype).eps / 2
    for name, got, want in zip(("x", "w", "b", "table"), _library(p, m), _autograd(p, m)):
        err = (got.double() - want).norm() / want.norm()
        assert err < bound, (name, err.item(), bound)


def test_calls_on_two_streams_at_once():
    """Calls that overlap on the GPU, each with its own inputs and workspace,
    give the bits that they give alone."""
    gen = torch.Generator(DEV).manual_seed(3)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)
    bucket = wgs.build_window_buckets((1, 7, 7), device=DEV)
    small = wgs.build_window_buckets((1, 3, 3), device=DEV)
    plan, plan3 = wgs.build_bucket_plan(bucket, 169, device=DEV), wgs.build_bucket_plan(small, 25, device=DEV)
    work = []
    for _ in range(2):
        x, gy, w, b = rand(3, 5000, 96), rand(3, 5000, 96), rand(96), rand(96)
        xs, table = rand(900, 30, 64).half(), rand(2, 169, 4)
        grad, grad3 = rand(300, 4, 49, 49).half(), rand(700, 6, 9, 9)
        types = torch.randint(0, 2, (300,), generator=gen, device=DEV, dtype=torch.int32)

        def run(x=x, gy=gy, w=w, b=b, xs=xs, table=table, grad=grad, grad3=grad3, types=types):
            y, mean, rstd = wgs.group_norm_act(x, 8, w, b, 1e-5, "silu")
            return (y, mean, rstd, *wgs.group_norm_act_bwd(gy, x, 8, mean, rstd, w, b, "silu"),
                    wgs.group_norm_act(xs, 16)[0], wgs.position_bias(table, bucket, torch.float16),
                    wgs.position_bias_bwd(grad, plan, types, 2), wgs.position_bias_bwd(grad3, plan3))
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
            for outs in each:
                assert all(torch.equal(p, q) for p, q in zip(outs, alone))
    wgs.check_error(DEV)
