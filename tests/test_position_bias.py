"""The learned position bias by buckets: host maps and plans, the expansion
(bit-exact against the oracle) and the table's gradient.

Tolerance of the gradient.  It is an FP32 sum of gradients in a fixed order:
windows of a slab one after another, then a slot's pairs, then slots and
slabs over some lanes.  With D additions on the longest path and u = 2^-24 its error is at
most D u sum|g| (1 + small), and rounding to a 16-bit table adds half a step.
D <= windows + 4096 (a tile's pairs) + tiles * slabs; 64 slabs bound every
case here.
"""
import ctypes
import dataclasses
import itertools

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
A, B, C, D, E = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000


def _np(t, fmt):
    t = t.detach().cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if fmt == "bf16" else t.numpy()


def _values(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------- host: the maps ----

@pytest.mark.parametrize("window", [(1, 1, 1), (2, 6, 12), (1, 7, 7), (3, 1, 5), (2, 3, 4)])
@pytest.mark.parametrize("absolute", range(8))
def test_window_buckets_equal_the_oracle(window, absolute):
    got = wgs.build_window_buckets(window, absolute).numpy()
    assert np.array_equal(got, oracle.build_window_buckets(window, absolute))
    count = wgs.window_bucket_count(window, absolute)
    assert got.min() == 0 and got.max() == count - 1
    if absolute == 0:   # the difference alone: i -> j and back mirror each other
        assert np.array_equal(got + got.T, np.full_like(got, count - 1))
    if absolute == 7:   # every pair has a bucket of its own
        assert len(np.unique(got)) == got.size


def test_window_buckets_worked():
    # 1 x 1 x 3 cells: bucket = i - j + 2; absolute: 3 i + j
    assert wgs.build_window_buckets((1, 1, 3)).tolist() == [[2, 1, 0], [3, 2, 1], [4, 3, 2]]
    assert wgs.build_window_buckets((1, 1, 3), 4).tolist() == [[0, 1, 2], [3, 4, 5], [6, 7, 8]]
    # the 144-cell window with depth and latitude absolute
    assert wgs.window_bucket_count((2, 6, 12), 3) == 4 * 36 * 23


@pytest.mark.parametrize("n_q,n_k,start,buckets,reach,both", [
    (1, 1, 0, 4, 3, True), (1, 200, 199, 32, 128, True), (65, 65, 0, 32, 128, False),
    (7, 300, 40, 8, 16, True), (33, 5, 0, 2, 9, False), (1, 40, 0, 16, 100, False),
    (40, 40, 0, 12, 20, True)])
def test_distance_buckets_equal_the_oracle(n_q, n_k, start, buckets, reach, both):
    got = wgs.build_distance_buckets(n_q, n_k, buckets, reach, both, start).numpy()
    assert np.array_equal(got, oracle.build_distance_buckets(n_q, n_k, buckets, reach, both, start))
    assert got.max() < buckets and got.min() >= (0 if both else -1)


def test_distance_buckets_worked():
    """32 buckets both ways, reach 128: 16 a direction, 8 of them single
    distances, then borders at 8 * 16^(k/8) = 8 * 2^(k/2)."""
    row = wgs.build_distance_buckets(1, 400, 32, 128, True, 200).numpy()[0]
    behind = {0: 0, 1: 1, 7: 7, 8: 8, 11: 8, 12: 9, 15: 9, 16: 10, 22: 10, 23: 11, 31: 11, 32: 12,
              64: 14, 90: 14, 91: 15, 127: 15, 128: 15, 199: 15}
    for d, b in behind.items():
        assert row[200 - d] == b, d
        if d:
            assert row[min(200 + d, 399)] == 16 + b, d


def test_map_builder_refusals():
    lib = _capi.load()
    w = (ctypes.c_int32 * 3)(2, 3, 4)
    out = (ctypes.c_int32 * 576)()
    f = lib.wgs_build_window_buckets
    assert f(w, 0, out, 576) == OK
    assert f(w, 0, out, 575) == SHAPE
    assert f(w, 8, out, 576) == SHAPE and f(w, -1, out, 576) == SHAPE
    assert f((ctypes.c_int32 * 3)(0, 3, 4), 0, out, 576) == SHAPE
    assert f((ctypes.c_int32 * 3)(40000, 40000, 1), 0, out, 2 ** 62) == SHAPE
    assert f(None, 0, out, 576) == NULL and f(w, 0, None, 576) == NULL
    assert lib.wgs_window_bucket_count((ctypes.c_int32 * 3)(46341, 1, 1), 1) == -1
    assert lib.wgs_window_bucket_count((ctypes.c_int32 * 3)(46340, 1, 1), 1) == 46340 ** 2
    g = lib.wgs_build_distance_buckets
    assert g(4, 4, 0, 32, 128, 1, out, 16) == OK
    assert g(4, 4, 0, 32, 128, 1, out, 15) == SHAPE
    assert g(4, 4, -1, 32, 128, 1, out, 16) == SHAPE
    assert g(-4, 4, 0, 32, 128, 1, out, 16) == SHAPE
    assert g(4, 4, 0, 31, 128, 1, out, 16) == SHAPE      # odd, both directions
    assert g(4, 4, 0, 1, 128, 0, out, 16) == SHAPE       # one bucket a direction
    assert g(4, 4, 0, 32, 8, 1, out, 16) == SHAPE        # reach no farther than single distances
    assert g(4, 4, 0, 32, 128, 2, out, 16) == SHAPE
    assert g(4, 4, 0, 32, 128, 1, None, 16) == NULL
    assert g(0, 4, 0, 32, 128, 1, None, 0) == OK
    assert g(2 ** 31 - 1, 2 ** 31 - 1, 0, 32, 128, 1, out, 576) == SHAPE


def test_distance_buckets_of_a_reach_beyond_all_pairs():
    # (the table of single distances is as long as the pairs need)
    got = wgs.build_distance_buckets(3, 5, 32, 2 ** 31 - 1, True, 2)
    d = np.arange(5)[None] - (np.arange(3)[:, None] + 2)
    assert np.array_equal(got.numpy(), np.abs(d) + 16 * (d > 0))      # all below 8
    assert np.array_equal(got.numpy(), oracle.build_distance_buckets(3, 5, 32, 2 ** 31 - 1, True, 2))


# ------------------------------------------------------- host: the plan ----

TILE = 4096


def _plan_parts(plan):
    """The sections of a plan by its documented layout: the lanes' bits and
    first slots, each bucket's slots, and the order, lane by lane."""
    w = plan.words.cpu().numpy()
    up = lambda v: (v + 3) // 4 * 4
    tiles = -(-plan.n_pairs // TILE)
    assert w[:5].tolist() == [0x57425032, plan.n_pairs, plan.n_buckets, tiles, plan.n_slots]
    at = 8
    parts = []
    for n in (tiles * 256, plan.n_buckets + 1, plan.n_slots):
        parts.append(w[at:at + n])
        at += up(n)
    order = w[at:].view(np.uint16).reshape(tiles, 4, 128, 8).transpose(0, 2, 1, 3).reshape(tiles, TILE)
    order = order ^ (order >> 5 & 31)      # places of the sums back to pairs
    lane = parts[0].reshape(tiles, 128, 2)
    return lane[..., 0].view(np.uint32), lane[..., 1], parts[1], parts[2], order


def _maps():
    rng = np.random.default_rng(5)
    yield wgs.build_window_buckets((2, 6, 12), 3), wgs.window_bucket_count((2, 6, 12), 3)
    yield wgs.build_window_buckets((1, 7, 7)), 169
    yield wgs.build_distance_buckets(70, 130, 32, 128, False), 32
    yield torch.full((3, 5), -1, dtype=torch.int32), 4
    yield torch.zeros(1, 1, dtype=torch.int32), 1
    yield torch.zeros(0, 7, dtype=torch.int32), 3
    yield torch.zeros(90, 91, dtype=torch.int32), 2
    yield torch.from_numpy(rng.integers(-1, 5000, (80, 113)).astype(np.int32)), 5000


@pytest.mark.parametrize("i", range(8))
def test_plan_inverts_its_map(i):
    bucket, n_buckets = next(itertools.islice(_maps(), i, None))
    plan = wgs.build_bucket_plan(bucket, n_buckets, device="cpu")
    ends, first_slot, bucket_first, bucket_slot, order = _plan_parts(plan)
    flat = bucket.numpy().reshape(-1)
    assert sorted(bucket_slot.tolist()) == list(range(plan.n_slots))
    of_slot = np.full(plan.n_slots, -1)
    for b in range(plan.n_buckets):
        mine = bucket_slot[bucket_first[b]:bucket_first[b + 1]]
        assert (np.diff(mine) > 0).all()
        of_slot[mine] = b
    # a slot is a run of a lane's entries up to a set bit: each pair once, in
    # the slot of its bucket, slots numbered along the order
    seen = np.full(flat.size, -1)
    expect = 0
    for t in range(len(ends)):
        for l in range(128):
            slot, begin = first_slot[t, l], 0
            for e in range(32):
                if not ends[t, l] >> e & 1:
                    continue
                assert slot == expect
                pairs = t * TILE + order[t, 32 * l + begin:32 * l + e + 1].astype(np.int64)
                assert (np.diff(pairs) > 0).all() and (seen[pairs] == -1).all()
                seen[pairs] = of_slot[slot]
                slot, begin, expect = slot + 1, e + 1, expect + 1
    assert expect == plan.n_slots
    assert np.array_equal(seen, flat)


def test_plan_refusals():
    lib = _capi.load()
    m = (ctypes.c_int32 * 4)(0, 1, -1, 2)
    bad = (ctypes.c_int32 * 4)(0, 1, -2, 2)
    n = ctypes.c_int64()
    words = lib.wgs_bucket_plan_words(m, 4, 3, ctypes.byref(n))
    assert words > 0 and n.value == 3
    out = (ctypes.c_int32 * words)()
    assert lib.wgs_build_bucket_plan(m, 4, 3, out, words) == OK
    assert lib.wgs_build_bucket_plan(m, 4, 3, out, words - 1) == SHAPE
    assert lib.wgs_build_bucket_plan(m, 4, 2, out, words) == INDEX
    assert lib.wgs_build_bucket_plan(bad, 4, 3, out, words) == INDEX
    assert lib.wgs_build_bucket_plan(None, 4, 3, out, words) == NULL
    assert lib.wgs_build_bucket_plan(m, 4, 3, None, words) == NULL
    assert lib.wgs_build_bucket_plan(m, -1, 3, out, words) == SHAPE
    assert lib.wgs_bucket_plan_words(bad, 4, 3, None) == -1
    assert lib.wgs_bucket_plan_words(m, 4, 0, None) == -1
    assert lib.wgs_bucket_plan_words(m, 2 ** 31, 3, None) == -1
    with pytest.raises(RuntimeError, match="bucket values"):
        wgs.build_bucket_plan(torch.tensor([[3]], dtype=torch.int32), 3, device="cpu")
    with pytest.raises(RuntimeError, match="int32"):
        wgs.build_bucket_plan(torch.tensor([[1]]), 3, device="cpu")


# -------------------------------------------------- refusals of the calls ----

def test_position_bias_refusals():
    """Every call here is refused while its arguments are checked."""
    f = _capi.load().position_bias
    # (table, bucket, bias, n_types, heads, n_pairs, n_buckets, table_dtype, dtype, stream)
    assert f(A, B, C, 1, 6, 144, 9, 3, 1, None) == DTYPE
    assert f(A, B, C, 1, 6, 144, 9, 1, 2, None) == DTYPE        # fp16 table, bf16 bias
    assert f(A, B, C, 1, 6, 144, 9, 1, 0, None) == DTYPE        # fp16 table, fp32 bias
    assert f(A, B, C, -1, 6, 144, 9, 0, 1, None) == SHAPE
    assert f(A, B, C, 1, 6, 144, 0, 0, 1, None) == SHAPE        # pairs, but no bucket
    assert f(A, B, C, 1, 6, 2 ** 31, 9, 0, 1, None) == SHAPE
    assert f(A, B, C, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 30, 9, 0, 1, None) == SHAPE
    assert f(None, None, None, 0, 6, 144, 9, 0, 1, None) == OK
    assert f(None, None, None, 1, 6, 0, 0, 0, 1, None) == OK
    for k in range(3):
        p = [A, B, C]
        p[k] = None
        assert f(*p, 1, 6, 144, 9, 0, 1, None) == NULL
    assert f(A + 2, B, C, 1, 6, 144, 9, 0, 1, None) == ALIGN
    assert f(A, B + 2, C, 1, 6, 144, 9, 0, 1, None) == ALIGN
    assert f(A, B, C + 1, 1, 6, 144, 9, 0, 1, None) == ALIGN
    assert f(A, B, A + 64, 1, 6, 144, 9, 0, 1, None) == ALIAS
    assert f(A, C + 64, C, 1, 6, 144, 9, 0, 1, None) == ALIAS


def test_position_bias_bwd_refusals():
    lib = _capi.load()
    f = lib.position_bias_bwd
    need = lib.wgs_position_bias_bwd_workspace_bytes(4, 6, 1, 144, 20)
    assert need == 6 * 20 * 4
    assert lib.wgs_position_bias_bwd_workspace_bytes(-1, 6, 1, 144, 20) == 0

    def call(grad=A, plan=B, types=None, out=C, ws=D, ws_bytes=need, n_win=4, heads=6, n_pairs=144,
             buckets=9, slots=20, n_types=1, dtype=1, table=0):
        return f(grad, plan, types, out, ws, ws_bytes, n_win, heads, n_pairs, buckets, slots,
                 n_types, dtype, table, None)

    assert call(dtype=4) == DTYPE and call(table=2) == DTYPE
    assert call(n_win=-1) == SHAPE and call(slots=-1) == SHAPE and call(slots=145) == SHAPE
    assert call(n_pairs=2 ** 31) == SHAPE
    assert call(n_types=2 ** 31 - 1, heads=2 ** 31 - 1) == SHAPE
    assert call(ws_bytes=need - 1) == SHAPE
    assert call(grad=None) == NULL and call(plan=None) == NULL and call(out=None) == NULL
    assert call(ws=None) == NULL
    assert call(grad=A + 1) == ALIGN and call(plan=B + 4) == ALIGN and call(types=E + 2) == ALIGN
    assert call(out=C + 2) == ALIGN and call(ws=D + 8) == ALIGN
    assert call(out=A + 64) == ALIAS and call(ws=A + 64) == ALIAS and call(out=B + 16) == ALIAS
    assert call(ws=B + 16) == ALIAS and call(out=D + 16) == ALIAS
    assert call(types=C + 4) == ALIAS and call(types=D + 4) == ALIAS
    assert call(grad=None, plan=None, out=None, ws=None, n_types=0) == OK
    assert call(grad=None, plan=None, out=None, ws=None, heads=0) == OK
    assert call(grad=None, plan=None, out=None, ws=None, buckets=0) == OK


def test_position_bias_bwd_refuses_too_many_windows():
    f = _capi.load().position_bias_bwd
    # the workspace is said to be large enough; nothing is launched
    args = (A, B, None, C, D, 2 ** 62)
    assert f(*args, 2 ** 31 - 65536, 1, 1, 1, 1, 1, 0, 0, None) == SHAPE
    assert f(*args, 2 ** 31 - 65536, 1, 144, 9, 20, 1, 1, 0, None) == SHAPE


def test_python_refusals_on_the_cpu():
    t, b = torch.zeros(1, 4, 2), torch.zeros(3, 3, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="CUDA"):
        wgs.position_bias(t, b)
    plan = wgs.build_bucket_plan(b, 4, device="cpu")
    with pytest.raises(RuntimeError, match="CUDA"):
        wgs.position_bias_bwd(torch.zeros(1, 2, 3, 3), plan)
    assert wgs.position_bias_bwd_workspace_bytes(plan, 5, 2) == 2 * 4


# --------------------------------------------------------- GPU: forward ----

FWD = [  # map, buckets, types, heads
    (lambda: wgs.build_window_buckets((2, 6, 12), 3), 3312, 3, 6),
    (lambda: wgs.build_window_buckets((2, 6, 12)), 759, 1, 12),
    (lambda: wgs.build_window_buckets((1, 7, 7)), 169, 2, 3),
    (lambda: wgs.build_window_buckets((1, 1, 1)), 1, 1, 1),
    (lambda: wgs.build_window_buckets((1, 2, 3), 2), 20, 5, 7),
    (lambda: wgs.build_distance_buckets(1, 1000, 32, 128, True, 999), 32, 1, 16),
    (lambda: wgs.build_distance_buckets(1, 37, 8, 20, False, 20), 8, 1, 5),
    (lambda: wgs.build_distance_buckets(130, 260, 32, 128, False), 32, 1, 8),
    (lambda: wgs.build_distance_buckets(63, 65, 16, 50, True), 16, 2, 2),
    (lambda: torch.full((8, 8), -1, dtype=torch.int32), 3, 1, 4),
]
PAIRS = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]


def _table(n_types, n_buckets, heads, fmt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n_types, n_buckets, heads, generator=g).to(DT[fmt])


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def _check_forward(table, bucket, table_fmt, fmt, out=None):
    got = wgs.position_bias(table, bucket, dtype=DT[fmt], out=out)
    want, bad = oracle.position_bias(_np(table, table_fmt), bucket.cpu().numpy(), table_fmt, fmt)
    assert got.shape == want.shape and bad == 0
    assert np.array_equal(_np(_bits(got), "f32"), want.view(np.int32 if fmt == "f32" else np.int16))
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("table_fmt,fmt", PAIRS)
@pytest.mark.parametrize("i", range(len(FWD)))
def test_position_bias_is_bit_exact(i, table_fmt, fmt):
    make, n_buckets, n_types, heads = FWD[i]
    table = _table(n_types, n_buckets, heads, table_fmt, i).to(DEV)
    _check_forward(table, make().to(DEV), table_fmt, fmt)
    wgs.check_error(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("table_fmt,fmt", PAIRS)
@pytest.mark.parametrize("shift", [1, 3, 5])
def test_position_bias_on_unaligned_buffers(table_fmt, fmt, shift):
    """Outputs, tables and maps that start between 16-byte borders; what lies
    before and behind the output stays as it was."""
    bucket, n_buckets, n_types, heads = wgs.build_window_buckets((1, 4, 6)), 77, 3, 4
    table = _table(n_types, n_buckets, heads, table_fmt, shift)
    tbuf = torch.zeros(table.numel() + 8, dtype=table.dtype, device=DEV)
    tv = tbuf[shift:shift + table.numel()].view(table.shape)
    tv.copy_(table)
    mbuf = torch.zeros(bucket.numel() + 8, dtype=torch.int32, device=DEV)
    mv = mbuf[shift:shift + bucket.numel()].view(bucket.shape)
    mv.copy_(bucket)
    n = n_types * heads * bucket.numel()
    obuf = torch.full((n + 16,), 7.0, dtype=DT[fmt], device=DEV)
    out = obuf[shift:shift + n].view(n_types, heads, *bucket.shape)
    for t, b in ((tv, bucket.to(DEV)), (table.to(DEV), mv), (tv, mv)):
        _check_forward(t, b, table_fmt, fmt, out=out)
        _check_forward(t, b, table_fmt, fmt)
    assert (obuf[:shift] == 7.0).all() and (obuf[shift + n:] == 7.0).all()
    # a 2-D table is one type
    one = wgs.position_bias(table[0].to(DEV), bucket.to(DEV), dtype=DT[fmt])
    assert torch.equal(_bits(one[0]), _bits(wgs.position_bias(table.to(DEV), bucket.to(DEV),
                                                              dtype=DT[fmt])[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,n_k", [(4, 8), (3, 5)])
def test_position_bias_special_values_and_bad_buckets(n_q, n_k):
    special = torch.tensor([float("inf"), float("-inf"), float("nan"), 65504.0, 1e30, -0.0, 6e-8, 1e-30])
    table = special.view(1, 8, 1).repeat(1, 1, 2).to(DEV)
    bucket = (torch.arange(n_q * n_k, dtype=torch.int32) % 9 - 1).view(n_q, n_k)
    got = wgs.position_bias(table, bucket.to(DEV), dtype=torch.float16)
    want = torch.where(bucket >= 0, special[bucket.clamp(min=0).long()], 0.0).half()
    assert torch.equal(got[0, 1].cpu().isnan(), want.isnan())
    assert torch.equal(got[0, 1].cpu().nan_to_num(nan=1.0), want.nan_to_num(nan=1.0))
    wgs.check_error(DEV)
    bucket[1, 2], bucket[2, 3] = 8, -2
    got = wgs.position_bias(torch.ones(1, 8, 2, device=DEV), bucket.to(DEV))
    assert torch.equal(got[0, 0].cpu(), ((bucket >= 0) & (bucket < 8)).float())
    with pytest.raises(wgs.WgsError, match="WGS_ERR_INDEX"):
        wgs.check_error(DEV)
    wgs.check_error(DEV)          # cleared


@pytest.mark.gpu
def test_position_bias_empty():
    b = torch.zeros(0, 5, dtype=torch.int32, device=DEV)
    assert wgs.position_bias(torch.zeros(2, 3, 4, device=DEV), b).shape == (2, 4, 0, 5)
    b = torch.zeros(2, 5, dtype=torch.int32, device=DEV)
    assert wgs.position_bias(torch.zeros(2, 3, 0, device=DEV), b).shape == (2, 0, 2, 5)
    with pytest.raises(wgs.WgsError, match="WGS_ERR_SHAPE"):
        wgs.position_bias(torch.zeros(2, 0, 4, device=DEV), b)
    for table, bucket, kw in ((torch.zeros(2, 3, 4, device=DEV), b.long(), {}),
                              (torch.zeros(2, 3, 4, device=DEV).half(), b, {"dtype": torch.float32}),
                              (torch.zeros(3, device=DEV), b, {}),
                              (torch.zeros(4, 3, device=DEV).t(), b, {}),
                              (torch.zeros(2, 3, 4, device=DEV), b, {"out": torch.zeros(1, device=DEV)})):
        with pytest.raises(RuntimeError):
            wgs.position_bias(table, bucket, **kw)


# -------------------------------------------------------- GPU: backward ----

BWD = [  # map, buckets, types, heads, windows
    (lambda: wgs.build_window_buckets((2, 6, 12), 3), 3312, 4, 3, 61),
    (lambda: wgs.build_window_buckets((2, 6, 12)), 759, 1, 2, 30),
    (lambda: wgs.build_window_buckets((1, 7, 7)), 169, 3, 2, 100),
    (lambda: wgs.build_window_buckets((1, 1, 1)), 1, 1, 1, 1),
    (lambda: wgs.build_window_buckets((1, 2, 3), 2), 20, 5, 7, 9),
    (lambda: wgs.build_window_buckets((1, 4, 4)), 49, 2, 5, 1300),
    (lambda: wgs.build_distance_buckets(1, 1000, 32, 128, True, 999), 32, 1, 4, 3),
    (lambda: wgs.build_distance_buckets(130, 260, 32, 128, False), 32, 1, 3, 2),
    (lambda: wgs.build_distance_buckets(63, 65, 16, 50, True), 16, 2, 2, 12),
    (lambda: torch.full((8, 8), -1, dtype=torch.int32), 3, 1, 4, 5),
    (lambda: torch.zeros(65, 64, dtype=torch.int32), 1, 1, 1, 7),
]


def _grad(shape, fmt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(DT[fmt])


def _check_backward(grad, bucket, plan, win_type, n_types, fmt, table_fmt, **kw):
    got = wgs.position_bias_bwd(grad, plan, win_type, n_types, dtype=DT[table_fmt], **kw)
    types = None if win_type is None else win_type.cpu().numpy()
    want, mag = oracle.position_bias_bwd(_np(grad, fmt), bucket.numpy(), types, n_types,
                                         plan.n_buckets, fmt)
    depth = grad.shape[0] + TILE + 64 * -(-plan.n_pairs // TILE)
    half = torch.finfo(DT[table_fmt]).eps / 2
    tiny = torch.finfo(DT[table_fmt]).smallest_normal * half
    bound = depth * U * mag + half * np.abs(want) * (1 + depth * U) + tiny
    err = np.abs(_values(got) - want)
    assert got.shape == want.shape and (err <= bound).all(), (err - bound).max()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("table_fmt,fmt", PAIRS)
@pytest.mark.parametrize("order", ["none", "runs", "mixed"])
@pytest.mark.parametrize("i", range(len(BWD)))
def test_position_bias_gradient(i, order, table_fmt, fmt):
    make, n_buckets, n_types, heads, n_win = BWD[i]
    bucket = make()
    plan = wgs.build_bucket_plan(bucket, n_buckets, device=DEV)
    grad = _grad((n_win, heads) + tuple(bucket.shape), fmt, 31 * i).to(DEV)
    types = None
    if order == "runs":
        types = (torch.arange(n_win) * n_types // n_win).int().to(DEV)
    elif order == "mixed":
        types = torch.randint(0, n_types, (n_win,), generator=torch.Generator().manual_seed(i)).int().to(DEV)
    need = wgs.position_bias_bwd_workspace_bytes(plan, n_win, heads, n_types)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)   # NaN patterns
    got = _check_backward(grad, bucket, plan, types, n_types, fmt, table_fmt, workspace=ws)
    assert (ws[need:] == 0xff).all()
    again = wgs.position_bias_bwd(grad, plan, types, n_types, dtype=DT[table_fmt])
    assert torch.equal(_bits(got), _bits(again))        # a fixed order of additions
    wgs.check_error(DEV)


# Maps of few pairs: windows shared out over groups of threads, several heads a
# block (the last with fewer), maps that just do and just do not belong here.
FEW = [  # map, buckets, types, heads, windows
    (lambda: wgs.build_window_buckets((1, 1, 1)), 1, 3, 32, 4096),
    (lambda: wgs.build_window_buckets((1, 2, 2)), 9, 1, 5, 777),
    (lambda: wgs.build_window_buckets((1, 3, 3)), 25, 4, 100, 90),
    (lambda: wgs.build_distance_buckets(16, 16, 8, 10, False), 8, 2, 12, 333),
    (lambda: wgs.build_window_buckets((1, 4, 8)), 105, 2, 7, 150),
    (lambda: wgs.build_distance_buckets(31, 33, 32, 20), 32, 1, 9, 60),
    (lambda: wgs.build_distance_buckets(25, 41, 32, 20), 32, 1, 9, 60),
    (lambda: wgs.build_window_buckets((1, 1, 2)), 3, 70, 1, 5000),
    (lambda: torch.full((3, 7), -1, dtype=torch.int32), 2, 1, 3, 40),
]


@pytest.mark.gpu
@pytest.mark.parametrize("table_fmt,fmt", [("f32", "f32"), ("f32", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("i", range(len(FEW)))
def test_gradient_of_small_maps(i, table_fmt, fmt):
    make, n_buckets, n_types, heads, n_win = FEW[i]
    bucket = make()
    plan = wgs.build_bucket_plan(bucket, n_buckets, device=DEV)
    buf = _grad((n_win * heads * bucket.numel() + 3,), fmt, i).to(DEV)
    grad = buf[:-3].view((n_win, heads) + tuple(bucket.shape))
    types = torch.randint(0, n_types, (n_win,), generator=torch.Generator().manual_seed(i)).int().to(DEV)
    got = _check_backward(grad, bucket, plan, types if n_types > 1 else None, n_types, fmt, table_fmt)
    # elsewhere in memory, the same bits
    view = torch.cat([buf[:1], buf[:-3]])[1:].view(grad.shape)
    again = wgs.position_bias_bwd(view, plan, types if n_types > 1 else None, n_types, dtype=DT[table_fmt])
    assert torch.equal(_bits(got), _bits(again))
    # without types every window counts for the first
    first = _check_backward(grad, bucket, plan, None, n_types, fmt, table_fmt)
    assert not first[1:].any()
    wgs.check_error(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_gradient_of_unaligned_views_equals_the_aligned_one(fmt):
    """The 16-byte and the element path add in the same order."""
    bucket = wgs.build_window_buckets((1, 4, 6))
    plan = wgs.build_bucket_plan(bucket, 77, device=DEV)
    grad = _grad((9, 3, 24, 24), fmt, 8).to(DEV)
    buf = torch.zeros(grad.numel() + 8, dtype=grad.dtype, device=DEV)
    view = buf[1:1 + grad.numel()].view(grad.shape)
    view.copy_(grad)
    a = _check_backward(grad, bucket, plan, None, 1, fmt, "f32")
    b = _check_backward(view, bucket, plan, None, 1, fmt, "f32")
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_gradient_edges():
    bucket = wgs.build_window_buckets((1, 2, 4))
    plan = wgs.build_bucket_plan(bucket, 21, device=DEV)
    # no windows: zeros, also over an output that held something else
    out = torch.full((2, 21, 3), 5.0, device=DEV)
    wgs.position_bias_bwd(torch.zeros(0, 3, 8, 8, device=DEV), plan, None, 2, grad_table=out)
    assert (out == 0).all()
    # no pairs
    none = wgs.build_bucket_plan(torch.zeros(0, 4, dtype=torch.int32), 21, device=DEV)
    assert (wgs.position_bias_bwd(torch.zeros(5, 3, 0, 4, device=DEV), none) == 0).all()
    # NaN and infinity reach their own bucket and head alone
    grad = torch.ones(2, 3, 8, 8, device=DEV)
    grad[1, 1, 0, 0] = float("nan")
    grad[0, 2, 0, 1] = float("inf")
    got = wgs.position_bias_bwd(grad, plan).cpu()
    b0, b1 = int(bucket[0, 0]), int(bucket[0, 1])
    assert got[0, b0, 1].isnan() and got[0, b1, 2] == float("inf")
    got[0, b0, 1] = got[0, b1, 2] = 0.0
    assert got.isfinite().all()
    # NaN in pairs without a bucket reaches nothing
    causal = wgs.build_distance_buckets(16, 16, 4, 8, False)
    grad = torch.ones(1, 1, 16, 16, device=DEV)
    grad[0, 0][causal.to(DEV) < 0] = float("nan")
    got = wgs.position_bias_bwd(grad, wgs.build_bucket_plan(causal, 4, device=DEV))
    assert got.sum().item() == 16 * 17 / 2
    wgs.check_error(DEV)


@pytest.mark.gpu
def test_gradient_reports_bad_types_and_foreign_plans():
    bucket = wgs.build_window_buckets((1, 2, 4))
    plan = wgs.build_bucket_plan(bucket, 21, device=DEV)
    grad = torch.ones(4, 2, 8, 8, device=DEV)
    types = torch.tensor([0, 2, 1, -1], dtype=torch.int32, device=DEV)
    got = wgs.position_bias_bwd(grad, plan, types, 2)
    want = torch.bincount(bucket.view(-1).long(), minlength=21).float()
    assert torch.equal(got.cpu(), want.view(1, 21, 1).expand(2, 21, 2))
    with pytest.raises(wgs.WgsError, match="WGS_ERR_INDEX"):
        wgs.check_error(DEV)
    # a plan built for other sizes: nothing of it is followed
    wrong = dataclasses.replace(plan, n_buckets=22)
    assert (wgs.position_bias_bwd(grad, wrong, None, 1) == 0).all()
    with pytest.raises(wgs.WgsError, match="WGS_ERR_INDEX"):
        wgs.check_error(DEV)
    for bad in (dict(win_type=types[:3]), dict(win_type=types.long()), dict(dtype=torch.float16),
                dict(workspace=torch.zeros(4, device=DEV)), dict(grad_table=torch.zeros(1, device=DEV))):
        with pytest.raises(RuntimeError):
            wgs.position_bias_bwd(grad, plan, **bad)
    with pytest.raises(RuntimeError, match="grad must be"):
        wgs.position_bias_bwd(torch.ones(4, 2, 8, 9, device=DEV), plan)
    with pytest.raises(wgs.WgsError, match="WGS_ERR_SHAPE"):
        wgs.position_bias_bwd(grad, plan, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))


@pytest.mark.gpu
def test_gradient_against_differences():
    """The expansion is linear in the table, so the difference of the scalar
    sum(grad * bias) under a step of one table entry is the gradient times
    the step; small integers make both exact in FP32."""
    bucket = wgs.build_window_buckets((1, 3, 4))
    n_buckets = wgs.window_bucket_count((1, 3, 4))
    plan = wgs.build_bucket_plan(bucket, n_buckets, device=DEV)
    g = torch.Generator().manual_seed(3)
    grad = torch.randint(-4, 5, (2, 2, 12, 12), generator=g).float().to(DEV)
    types = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    got = wgs.position_bias_bwd(grad, plan, types, 2)

    def value(table):
        return (wgs.position_bias(table, bucket.to(DEV))[types.long()] * grad).double().sum().item()

    base = torch.zeros(2, n_buckets, 2, device=DEV)
    for t, b, h in itertools.product(range(2), range(0, n_buckets, 5), range(2)):
        step = base.clone()
        step[t, b, h] = 1.0
        assert value(step) - value(base) == got[t, b, h].item()


@pytest.mark.gpu
def test_graph_replay_and_streams_give_the_same_bits():
    bucket = wgs.build_window_buckets((2, 3, 4))
    n_buckets = wgs.window_bucket_count((2, 3, 4))
    plan = wgs.build_bucket_plan(bucket, n_buckets, device=DEV)
    dbucket = bucket.to(DEV)
    grad = _grad((40, 4, 24, 24), "f16", 1).to(DEV)
    types = (torch.arange(40) % 3).int().to(DEV)
    table = _table(3, n_buckets, 4, "f32", 2).to(DEV)
    ws = [torch.empty(wgs.position_bias_bwd_workspace_bytes(plan, 40, 4, 3), dtype=torch.uint8,
                      device=DEV) for _ in range(2)]
    want = wgs.position_bias_bwd(grad, plan, types, 3), wgs.position_bias(table, dbucket, torch.float16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            wgs.position_bias_bwd(grad, plan, types, 3, grad_table=out[0], workspace=ws[0])
            wgs.position_bias(table, dbucket, out=out[1])
    other = torch.zeros_like(want[0])
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            graph.replay()
        wgs.position_bias_bwd(grad, plan, types, 3, grad_table=other, workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(other, want[0])
        assert torch.equal(_bits(out[1]), _bits(want[1]))
        for o in out:
            o.zero_()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [7400, 7401])
def test_offsets_past_32_bits(n):
    """More than 2^31 logits, in whole 16-byte runs and in odd rows: the last
    heads' bias and gradient."""
    heads, buckets = 40, 64
    bucket = wgs.build_distance_buckets(n, n, buckets, 4000, True)
    dbucket = bucket.to(DEV)
    assert heads * bucket.numel() > 2 ** 31
    table = _table(1, buckets, heads, "bf16", 3).to(DEV)
    bias = wgs.position_bias(table, dbucket)
    for h in (0, 19, 38, 39):
        assert torch.equal(_bits(bias[0, h]), _bits(table[0, :, h][dbucket.long()])), h
    # the bias itself as the gradient of one window
    plan = wgs.build_bucket_plan(bucket, buckets, device=DEV)
    got = wgs.position_bias_bwd(bias, plan)
    count = torch.bincount(dbucket.view(-1), minlength=buckets).double()
    want = table[0].double() * count[:, None]
    # a bucket's values are equal here, so its sum of magnitudes is |want|; pairs
    # are added over at most 4096 + 13372 tiles' slots
    assert ((got[0].double() - want).abs() <= 20000 * U * want.abs()).all()
    wgs.check_error(DEV)


@pytest.mark.gpu
def test_calls_with_given_outputs_allocate_nothing():
    bucket = wgs.build_window_buckets((1, 4, 6))
    plan, dbucket = wgs.build_bucket_plan(bucket, 77, device=DEV), bucket.to(DEV)
    table, grad = _table(2, 77, 4, "f32", 1).to(DEV), _grad((30, 4, 24, 24), "f16", 2).to(DEV)
    types = (torch.arange(30) % 2).int().to(DEV)
    out = torch.empty(2, 4, 24, 24, dtype=torch.float16, device=DEV)
    gt = torch.empty(2, 77, 4, device=DEV)
    ws = torch.empty(wgs.position_bias_bwd_workspace_bytes(plan, 30, 4, 2), dtype=torch.uint8, device=DEV)

    def calls():
        wgs.position_bias(table, dbucket, out=out)
        wgs.position_bias_bwd(grad, plan, types, 2, grad_table=gt, workspace=ws)

    calls()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    allocated, free = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0]
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == allocated
    assert torch.cuda.mem_get_info()[0] == free
