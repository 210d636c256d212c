"""Group norm as the first call of a process, at sizes whose shared memory
lies just at the 48 KB that a kernel gets without asking.

A kernel's own static shared memory counts towards that limit, and a raised
limit stays for the process, so each size has to be some kernel's first.  The
sizes: 49105 ... 49152 bytes asked for at launch, beside 48 static ones (some of
the forward's before its second pass kept a count a thread, and some since).
"""
import os
import subprocess
import sys

import pytest
import torch

import window_gather_swin_gb300 as wgs
from test_group_norm import DEV, _check_backward, _check_forward, _inputs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# n, spatial, channels, groups; format; activation: no two share a kernel
FORWARD = [
    ((1, 1000, 1024, 32), "f32", "silu"), ((1, 1000, 2048, 32), "f16", "gelu_tanh"),
    ((1, 1000, 2048, 8), "bf16", None), ((2, 300, 1146, 2), "f32", "gelu_tanh"),
    ((2, 300, 1726, 1726), "f16", None), ((700, 50, 592, 2), "f16", "silu"),
    ((2, 300, 832, 8), "f32", "gelu_tanh"), ((2, 300, 954, 2), "f32", None),
    ((700, 50, 832, 8), "bf16", "silu"), ((2, 300, 1630, 1630), "f16", "gelu_tanh"),
]
BACKWARD = [
    ((2, 300, 534, 534), "f32", None), ((1, 1000, 646, 2), "f32", "silu"),
    ((1, 1000, 1530, 2), "f16", "gelu_tanh"), ((700, 50, 664, 1), "f32", "gelu_tanh"),
    ((2, 300, 1535, 1535), "bf16", "silu"),
]

SCRIPT = """
import sys
sys.path.insert(0, {root!r})
import torch, window_gather_swin_gb300 as wgs
DT = {{"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}}
for (n, s, c, g), fmt, act in {forward!r}:
    x = torch.randn(n, s, c, device="cuda").to(DT[fmt])
    w, b = torch.ones(c, device="cuda"), torch.zeros(c, device="cuda")
    wgs.group_norm_act(x, g, w, b, 1e-5, act)
for (n, s, c, g), fmt, act in {backward!r}:
    x = torch.randn(n, s, c, device="cuda").to(DT[fmt])
    w, b = torch.ones(c, device="cuda"), torch.zeros(c, device="cuda")
    mean, rstd = torch.zeros(n, g, device="cuda"), torch.ones(n, g, device="cuda")
    wgs.group_norm_act_bwd(x, x, g, mean, rstd, w, b, act)
wgs.check_error()
"""


def _fresh(forward, backward):
    """The calls in a process of their own."""
    code = SCRIPT.format(root=ROOT, forward=forward, backward=backward)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-1500:]


@pytest.mark.gpu
def test_forward_at_the_shared_memory_limit():
    _fresh(FORWARD, [])
    for shape, fmt, act in FORWARD:
        x, w, b, _ = (t.to(DEV) for t in _inputs(shape, fmt, "f32", 3))
        _check_forward(x, w, b, shape[3], 1e-5, act, fmt)
    wgs.check_error(DEV)


@pytest.mark.gpu
def test_backward_at_the_shared_memory_limit():
    _fresh([], BACKWARD)
    for shape, fmt, act in BACKWARD:
        x, w, b, gy = (t.to(DEV) for t in _inputs(shape, fmt, "f32", 4))
        _, mean, rstd = wgs.group_norm_act(x, shape[3], w, b, 1e-5, act)
        _check_backward(gy, x, w, b, shape[3], mean, rstd, act, fmt, "f32")
    wgs.check_error(DEV)
