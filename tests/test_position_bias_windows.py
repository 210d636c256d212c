"""The position bias' gradient over many windows, against 64 bits.

Tolerance.  At most 128 windows are added to one FP32 register in a row and
the 128s to a second one, which a list of windows of one type, at most 1024
at a time, also ends; then come a lane's 32 pairs and the bucket's slots of
all slabs.  With u = 2^-24 and D = 256 + windows / 64 + slots the error is at
most D u times the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle
import window_gather_swin_gb300 as wgs

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16}

pytestmark = pytest.mark.gpu


def _slots(plan):
    """Slots of the bucket that has most."""
    w = plan.words.cpu().numpy()
    at = 8 + 256 * -(-plan.n_pairs // 4096)
    return int(np.diff(w[at:at + plan.n_buckets + 1]).max())


def _depth(plan, n_win, heads, n_types):
    slabs = wgs.position_bias_bwd_workspace_bytes(plan, n_win, heads, n_types) // (
        4 * n_types * heads * plan.n_slots)
    return 256 + n_win / 64 + _slots(plan) * slabs, slabs


@pytest.mark.parametrize("fmt", ["f32", "f16"])
@pytest.mark.parametrize("n_win", [1024, 1025, 1100, 2049])
@pytest.mark.parametrize("order", ["mixed", "runs", "halves"])
def test_types_of_more_windows_than_a_list_holds(n_win, order, fmt):
    """One slab of more windows than are looked over at a time: types without
    a window in a piece, in the last piece, or in any."""
    heads, n_types = 6, 50
    bucket = wgs.build_window_buckets((1, 7, 7))
    plan = wgs.build_bucket_plan(bucket, 169, device=DEV)
    gen = torch.Generator().manual_seed(n_win)
    if order == "runs":
        types = torch.arange(n_win) * n_types // n_win
    else:
        types = torch.randint(0, n_types, (n_win,), generator=gen)
        types[types == 7] = 8                       # none of type 7 ...
        if order == "halves":
            types[:1024] -= types[:1024] % 2        # ... and odd ones behind the first piece alone
    types = types.int()
    grad = (0.25 + torch.randn(n_win, heads, 49, 49, generator=gen)).to(DT[fmt])
    D, slabs = _depth(plan, n_win, heads, n_types)
    assert slabs == 1
    got = wgs.position_bias_bwd(grad.to(DEV), plan, types.to(DEV), n_types)
    wgs.check_error(DEV)
    want, mag = oracle.position_bias_bwd(grad.numpy(), bucket.numpy(), types.numpy(), n_types, 169, fmt)
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= (D + 1) * U * mag).all(), (err / np.maximum(mag * D * U, 1e-300)).max()
    assert order == "runs" or not got[7].any()


MANY = [  # map, buckets, heads, types (all windows have one), windows; units of one slab fill the GPU
    (lambda: wgs.build_distance_buckets(33, 33, 32, 128), 32, 1, 274, 20000),        # a tile each
    (lambda: wgs.build_distance_buckets(33, 34, 32, 128), 32, 1, 280, 6000),         # pairs in whole words
    (lambda: wgs.build_distance_buckets(35, 33, 32, 128), 32, 1, 280, 6000),         # odd pairs
    (lambda: wgs.build_distance_buckets(4, 4, 8, 16), 8, 32, 300, 60000),            # a small map
    (lambda: wgs.build_distance_buckets(20, 25, 8, 16), 8, 5, 300, 6000),
    (lambda: wgs.build_distance_buckets(1, 1, 8, 16), 8, 128, 200, 60000),
]


@pytest.mark.parametrize("typed", [True, False])
@pytest.mark.parametrize("fmt", ["f32", "f16"])
@pytest.mark.parametrize("i", range(len(MANY)))
def test_long_sums_of_equal_values(i, fmt, typed):
    """Gradients that are all 0.1: a running FP32 sum rounds the same way
    again and again, so that what its length costs shows."""
    make, n_buckets, heads, n_types, n_win = MANY[i]
    bucket = make()
    plan = wgs.build_bucket_plan(bucket, n_buckets, device=DEV)
    grad = torch.full((n_win, heads) + tuple(bucket.shape), 0.1, dtype=DT[fmt], device=DEV)
    types = torch.zeros(n_win, dtype=torch.int32, device=DEV) if typed else None
    got = wgs.position_bias_bwd(grad, plan, types, n_types)
    wgs.check_error(DEV)
    D, slabs = _depth(plan, n_win, heads, n_types)
    assert slabs == 1
    want = torch.bincount(bucket.view(-1), minlength=n_buckets).double() * n_win * grad[0, 0, 0, 0].item()
    err = (got[0].cpu().double() - want[:, None]).abs()
    assert (err <= D * U * want[:, None]).all(), (err / want[:, None]).max()
    assert not got[1:].any()


@pytest.mark.parametrize("fmt", ["f32", "f16"])
@pytest.mark.parametrize("shape", [(1500, 5, 20, 25), (700, 3, 33, 40), (3000, 3, 4, 6)])
def test_long_sums_elsewhere_in_memory_give_the_same_bits(shape, fmt):
    """Windows of a thread beyond one run of 128, with types and without, read
    in 16 bytes, words and elements."""
    n_win, heads, n_q, n_k = shape
    bucket = wgs.build_distance_buckets(n_q, n_k, 32, 128)
    plan = wgs.build_bucket_plan(bucket, 32, device=DEV)
    gen = torch.Generator(DEV).manual_seed(n_win)
    grad = torch.randn(shape, generator=gen, device=DEV).to(DT[fmt])
    buf = torch.zeros(grad.numel() + 8, dtype=grad.dtype, device=DEV)
    view = buf[1:1 + grad.numel()].view(shape)
    view.copy_(grad)
    types = torch.randint(0, 3, (n_win,), generator=gen, device=DEV, dtype=torch.int32)
    for t in (None, types, types * 0):
        a = wgs.position_bias_bwd(grad, plan, t, 300)
        assert torch.equal(a, wgs.position_bias_bwd(view, plan, t, 300))
        sums = torch.zeros(3, heads, n_q * n_k, dtype=torch.float64, device=DEV)
        mag = torch.zeros_like(sums)
        kinds = torch.zeros(n_win, dtype=torch.long, device=DEV) if t is None else t.long()
        sums.index_add_(0, kinds, grad.double().view(n_win, heads, -1))
        mag.index_add_(0, kinds, grad.double().abs().view(n_win, heads, -1))
        want, size = (torch.zeros(3, heads, 32, dtype=torch.float64, device=DEV).index_add_(
            2, bucket.to(DEV).view(-1).long(), v).transpose(1, 2) for v in (sums, mag))
        D, _ = _depth(plan, n_win, heads, 300)
        assert ((a[:3].double() - want).abs() <= D * U * size).all()
    wgs.check_error(DEV)


def test_inputs_written_right_before_the_call():
    """The plan, the types, the gradient and the table written in place by the
    kernels and copies just before, again and again with other values: no
    launch of a call may read what was there earlier."""
    for n_q, n_k, heads, n_win, n_types in ((49, 49, 3, 200, 2), (12, 12, 4, 300, 3), (300, 300, 2, 2, 1),
                                            (128, 128, 2, 40, 3)):
        gen = torch.Generator().manual_seed(n_q)
        n_buckets = 64
        # the same pairs in other buckets: plans of one size
        base = wgs.build_distance_buckets(n_q, n_k, n_buckets, 200)
        maps = [((base.long() + 5 * k) % n_buckets).int() for k in range(4)]
        plans = [wgs.build_bucket_plan(m, n_buckets, device=DEV) for m in maps]
        assert len({p.n_slots for p in plans}) == 1
        srcs = [(p.words, m.to(DEV), torch.randn(n_win, heads, n_q, n_k, generator=gen).half().to(DEV),
                 torch.randint(0, n_types, (n_win,), generator=gen).int().to(DEV),
                 torch.randn(n_types, n_buckets, heads, generator=gen).to(DEV)) for p, m in zip(plans, maps)]
        now = [t.clone() for t in srcs[0]]
        plan = wgs.BucketPlan(now[0], plans[0].shape, n_buckets, plans[0].n_slots)
        torch.cuda.synchronize()
        got = []
        for _ in range(5):
            for src in srcs:
                for to, t in zip(now, src):
                    to.copy_(t)
                got.append((wgs.position_bias_bwd(now[2], plan, now[3], n_types),
                            wgs.position_bias(now[4], now[1], torch.float16)))
        torch.cuda.synchronize()
        for k, src in enumerate(srcs):
            want = (wgs.position_bias_bwd(src[2], plans[k], src[3], n_types),
                    wgs.position_bias(src[4], src[1], torch.float16))
            torch.cuda.synchronize()
            for r in range(5):
                assert all(torch.equal(p, q) for p, q in zip(got[4 * r + k], want)), (n_q, k, r)
        wgs.check_error(DEV)
