"""The second kernel of the position bias' gradient: each of its forms on grids
that start early and on larger ones that wait, against 64 bits, and replayed
in a graph with the plan and the gradient overwritten in between.

Tolerance: FP32 sums of at most 128 windows, their runs, 32 pairs, and a bucket's
slots: D = 256 + slots additions, D u of the sum of magnitudes, u = 2^-24.
"""
import numpy as np
import pytest
import torch

import oracle
import window_gather_swin_gb300 as wgs

DEV = "cuda:0"
U = 2.0 ** -24

pytestmark = pytest.mark.gpu


def _random_map(n_q, n_k, n_buckets, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.integers(-1, n_buckets, (n_q, n_k)).astype(np.int32))


FORMS = [  # map, buckets, types, heads, windows
    (lambda: _random_map(40, 41, 1000, 1), 1000, 8, 2, 9),       # a thread a bucket, 32 blocks
    (lambda: _random_map(40, 41, 1000, 2), 1000, 400, 2, 500),   # 1600 blocks
    (lambda: wgs.build_distance_buckets(50, 60, 64, 50), 64, 3, 8, 20),      # lanes a bucket
    (lambda: wgs.build_distance_buckets(50, 60, 64, 50), 64, 700, 8, 900),
    (lambda: wgs.build_distance_buckets(70, 60, 2, 50, False), 2, 5, 4, 20),    # a block a bucket
    (lambda: wgs.build_distance_buckets(70, 60, 2, 50, False), 2, 120, 4, 300),
    (lambda: torch.full((64, 65), -1, dtype=torch.int32), 3, 2, 2, 3),       # no slots at all
]


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_pass_two_of_small_and_large_grids(i):
    make, n_buckets, n_types, heads, n_win = FORMS[i]
    bucket = make()
    plan = wgs.build_bucket_plan(bucket, n_buckets, device=DEV)
    gen = torch.Generator().manual_seed(i)
    grad = (0.3 + torch.randn((n_win, heads) + tuple(bucket.shape), generator=gen)).half()
    types = torch.randint(0, n_types, (n_win,), generator=gen).int()
    got = wgs.position_bias_bwd(grad.to(DEV), plan, types.to(DEV), n_types)
    wgs.check_error(DEV)
    want, mag = oracle.position_bias_bwd(grad.numpy(), bucket.numpy(), types.numpy(), n_types, n_buckets, "f16")
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= (256 + plan.n_slots) * U * mag).all(), (err / np.maximum(mag, 1e-30)).max()


@pytest.mark.parametrize("n_q,n_k,heads,n_win,n_types", [(49, 49, 4, 60, 3), (12, 12, 4, 60, 3), (130, 131, 2, 3, 1)])
def test_replayed_with_other_plans_and_gradients(n_q, n_k, heads, n_win, n_types):
    n_buckets = 64
    base = wgs.build_distance_buckets(n_q, n_k, n_buckets, 200)
    plans = [wgs.build_bucket_plan(((base.long() + 7 * k) % n_buckets).int(), n_buckets, device=DEV)
             for k in range(3)]
    gen = torch.Generator(DEV).manual_seed(n_q)
    grads = [torch.randn(n_win, heads, n_q, n_k, generator=gen, device=DEV).half() for _ in plans]
    types = torch.randint(0, n_types, (n_win,), generator=gen, device=DEV, dtype=torch.int32)
    want = [wgs.position_bias_bwd(g, p, types, n_types) for g, p in zip(grads, plans)]
    plan = wgs.BucketPlan(plans[0].words.clone(), plans[0].shape, n_buckets, plans[0].n_slots)
    grad, out = grads[0].clone(), torch.zeros_like(want[0])
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(2):         # two calls one behind the other, as a step makes them
                wgs.position_bias_bwd(grad, plan, types, n_types, grad_table=out)
        got = []
        for r in range(9):
            plan.words.copy_(plans[r % 3].words)
            grad.copy_(grads[r % 3])
            graph.replay()
            got.append(out.clone())
    torch.cuda.synchronize()
    for r in range(9):
        assert torch.equal(got[r], want[r % 3]), r
    wgs.check_error(DEV)
