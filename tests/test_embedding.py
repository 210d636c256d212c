"""Embedding lookup with scaling, and its gradient by sorted indices, against
the definitions in double precision.

The lookup is one FP32 product and one rounding to the output's format, which
torch's elementwise operations do as well: the bits are equal.

The gradient's sums.  Indices of a sorted piece: a slot's (at most 64), the slots of
a piece (at most 256), every fourth or fewer of the pieces that a run reaches into (of
which there are at most 913, or indices / 64) and those sums (at most 32).  Of a tile,
where the table has few rows or the call few indices: all of the tile's, at most 2048,
one after another, and the tiles, of which there are at most 152, or indices / 2048.  So
with D = 2048 + 152 + 64 + 256 + 229 + indices / 256 + 32 additions, which covers both,
and u = 2^-24 the sum is off by D u of its terms' magnitudes, the product with scale by
u, and rounding to the
output's format by half a step.  Where all values are small whole numbers every
sum is exact, and the result has to be.
"""
import pytest
import torch

import window_gather_swin_gb300 as wgs
from window_gather_swin_gb300 import _capi, synth

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OK, NULL, SHAPE, WIDTH, ALIGN, DTYPE, ARCH, LAUNCH, INDEX, ALIAS = range(10)
PTR = [0x10000000 * k for k in range(1, 14)]
FORMATS = [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")]


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def _half_step(want, dtype):
    f = torch.finfo(dtype)
    return want.abs().clamp(min=f.smallest_normal) * (f.eps / 2)


# --------------------------------------------------------------- refusals ----

def test_embedding_refusals():
    """Every call here is refused while its arguments are checked."""
    lib = _capi.load()
    t, i, o = PTR[:3]

    def call(t=t, i=i, o=o, n=100, rows=50, width=64, tdtype=0, dtype=1):
        return lib.embedding(t, i, o, n, rows, width, 1.0, tdtype, dtype, None)

    assert call(dtype=3) == DTYPE and call(tdtype=2) == DTYPE and call(tdtype=1, dtype=0) == DTYPE
    assert call(width=0) == WIDTH and call(width=32769) == WIDTH
    assert call(n=-1) == SHAPE and call(rows=-1) == SHAPE and call(n=2 ** 31) == SHAPE and call(rows=2 ** 31) == SHAPE
    assert call(n=0, t=None, i=None, o=None) == OK
    assert call(t=None) == NULL and call(i=None) == NULL and call(o=None) == NULL
    assert call(t=t + 2) == ALIGN and call(o=o + 1) == ALIGN and call(i=i + 2) == ALIGN
    assert call(o=t + 64) == ALIAS and call(o=i) == ALIAS


def test_embedding_bwd_refusals():
    lib = _capi.load()
    g, i, t, ws = PTR[:4]
    need = lib.wgs_embedding_bwd_workspace_bytes(100, 50, 64)
    assert need > 0
    for bad in ((-1, 50, 64), (100, -1, 64), (100, 50, 0), (100, 50, 32769), (2 ** 31, 50, 64), (100, 2 ** 31, 64)):
        assert lib.wgs_embedding_bwd_workspace_bytes(*bad) == 0

    def call(g=g, i=i, t=t, ws=ws, size=need, n=100, rows=50, width=64, dtype=1, tdtype=0):
        return lib.embedding_bwd(g, i, t, ws, size, n, rows, width, 1.0, dtype, tdtype, None)

    assert call(dtype=-1) == DTYPE and call(tdtype=2) == DTYPE
    assert call(width=0) == WIDTH and call(width=40000) == WIDTH
    assert call(n=-1) == SHAPE and call(rows=-1) == SHAPE and call(size=need - 1) == SHAPE
    for name in ("g", "i", "t", "ws"):
        assert call(**{name: None}) == NULL, name
    assert call(g=None, i=None, t=None, ws=None, n=0, rows=0) == OK
    assert call(g=g + 1) == ALIGN and call(t=t + 2) == ALIGN and call(i=i + 1) == ALIGN and call(ws=ws + 8) == ALIGN
    assert call(t=g) == ALIAS and call(t=i) == ALIAS and call(ws=g + 16) == ALIAS and call(ws=t) == ALIAS
    assert call(ws=i) == ALIAS


def test_python_refuses_cpu_tensors():
    t, i = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="CUDA"):
        wgs.embedding(t, i)
    with pytest.raises(RuntimeError, match="CUDA"):
        wgs.embedding_bwd(t[:3], i, 4)
    assert wgs.embedding_bwd_workspace_bytes(3, 4, 8) > 0
    with pytest.raises(RuntimeError, match="at most"):
        wgs.embedding_bwd_workspace_bytes(3, 4, 2 ** 31)


# -------------------------------------------------------------------- GPU ----

def _indices(n, rows, kind, seed):
    """int32 [n]: "uniform", "skew" (a few rows take most), "one" (a single row),
    "none" (pads alone), "once" (every row once, then pads), "runs" (in order)."""
    gen = torch.Generator(DEV).manual_seed(seed)
    u = torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)
    if kind == "one":
        idx = torch.full((n,), rows // 2, device=DEV)
    elif kind == "none":
        idx = torch.full((n,), -1, device=DEV)
    elif kind == "once":
        idx = torch.full((n,), -1, device=DEV)
        some = min(n, rows)
        idx[torch.randperm(n, generator=gen, device=DEV)[:some]] = torch.randperm(rows, generator=gen, device=DEV)[:some]
    elif kind == "runs":
        idx = torch.arange(n, device=DEV) * rows // n
    elif kind == "skew":
        idx = (rows * u ** 6).long()
    else:
        idx = (rows * u).long()
    idx = idx.clamp(max=rows - 1)
    if kind in ("uniform", "skew"):
        idx = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.1, -1, idx)
    return idx.to(torch.int32)


SHAPES = [  # indices, rows of the table, width
    (1, 1, 1), (1, 5, 8), (7, 3, 16), (180, 366, 192), (33, 1, 40), (256, 255, 24), (257, 256, 65), (1000, 257, 96),
    (4096, 24, 192), (4097, 1000, 5), (5000, 70000, 12), (300, 2 ** 20, 3), (2049, 40, 771), (700, 90, 2048),
    (65, 11, 2056), (40, 9, 4100), (9000, 300, 1), (20000, 2, 384), (3000, 65535, 64), (131, 65536, 130),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,tfmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_lookup(shape, fmt, tfmt):
    n, rows, width = shape
    gen = torch.Generator(DEV).manual_seed(n)
    table = torch.randn(rows, width, generator=gen, device=DEV).to(DT[tfmt])
    idx = _indices(n, rows, "uniform", 1)
    for scale in (1.0, 1.7, -0.3):
        out = wgs.embedding(table, idx, scale, dtype=DT[fmt])
        want = (table.float()[idx.clamp(min=0).long()] * torch.tensor(scale, device=DEV)).to(DT[fmt])
        want[idx < 0] = 0
        assert torch.equal(_bits(out), _bits(want))
    wgs.check_error(DEV)


def _check_gradient(grad, idx, rows, scale, got):
    n, width = grad.shape
    keep = idx >= 0
    want = torch.zeros(rows, width, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    for lo in range(0, width, 256):
        g = grad[keep, lo:lo + 256].double()
        want[:, lo:lo + 256].index_add_(0, idx[keep].long(), g)
        mag[:, lo:lo + 256].index_add_(0, idx[keep].long(), g.abs())
    s = torch.tensor(scale, dtype=torch.float32).double().item()
    want *= s
    most = min(n, 2048) + 152 + 64 + 256 + 229 + n / 256 + 32
    tol = (most * U * abs(s) * mag + U * want.abs()) * (1 + torch.finfo(got.dtype).eps) + _half_step(want, got.dtype)
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    # nothing is added where no index points
    assert (got[torch.bincount(idx[keep].long(), minlength=rows) == 0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["uniform", "skew", "one", "none", "once", "runs"])
@pytest.mark.parametrize("fmt,tfmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient(shape, fmt, tfmt, kind):
    n, rows, width = shape
    idx = _indices(n, rows, kind, 2)
    gen = torch.Generator(DEV).manual_seed(n + 1)
    grad = torch.randn(n, width, generator=gen, device=DEV).to(DT[fmt])
    need = wgs.embedding_bwd_workspace_bytes(n, rows, width)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)
    table = torch.full((rows, width), float("nan"), dtype=DT[tfmt], device=DEV)
    got = wgs.embedding_bwd(grad, idx, rows, 1.7, DT[tfmt], grad_table=table, workspace=ws)
    assert (ws[need:] == 0xff).all()
    _check_gradient(grad, idx, rows, 1.7, got)
    assert torch.equal(_bits(got), _bits(wgs.embedding_bwd(grad, idx, rows, 1.7, DT[tfmt])))
    # whole numbers: exact sums (|sum| <= 8 * 20000 < 2^24; where the output holds
    # fewer bits, the exact sum rounded once)
    whole = torch.randint(-8, 9, (n, width), generator=gen, device=DEV).to(DT[fmt])
    want = torch.zeros(rows, width, dtype=torch.float64, device=DEV)
    want.index_add_(0, idx[idx >= 0].long(), whole[idx >= 0].double())
    got = wgs.embedding_bwd(whole, idx, rows, 1.0, DT[tfmt])
    assert torch.equal(got, want.float().to(DT[tfmt]))
    wgs.check_error(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,kind", [((131040, 24, 192), "uniform"), ((131040, 32768, 384), "skew"),
                                        ((131040, 32768, 64), "one"), ((300001, 77777, 33), "skew"),
                                        ((262145, 1, 8), "one"), ((700000, 500, 4), "uniform"),
                                        ((3000000, 2 ** 21, 2), "uniform"), ((262144, 2 ** 18, 16), "once"),
                                        ((131072, 2 ** 17 - 1, 24), "runs"), ((9000000, 2 ** 28, 1), "skew"),
                                        ((8500000, 3000, 2), "uniform"), ((131040, 27, 40), "skew"), ((131040, 26, 40), "skew"),
                                        ((131040, 53, 20), "uniform"), ((131040, 54, 20), "uniform"),
                                        ((5000, 1, 4100), "one"), ((311297, 3, 1027), "uniform"),
                                        ((20000, 2, 1), "none"), ((400000, 100, 33), "skew"), ((400000, 64, 72), "skew"),
                                        ((30001, 6, 8), "runs")], ids=str)
@pytest.mark.parametrize("fmt,tfmt", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32")])
def test_gradient_of_many_indices(shape, kind, fmt, tfmt):
    n, rows, width = shape
    idx = _indices(n, rows, kind, 3)
    gen = torch.Generator(DEV).manual_seed(4)
    grad = torch.randn(n, width, generator=gen, device=DEV).to(DT[fmt])
    got = wgs.embedding_bwd(grad, idx, rows, 0.5, DT[tfmt])
    _check_gradient(grad, idx, rows, 0.5, got)
    assert torch.equal(_bits(got), _bits(wgs.embedding_bwd(grad, idx, rows, 0.5, DT[tfmt])))
    # a row gets at most half a million terms of at most 2: sums below 2^24
    whole = torch.randint(-2, 3, (n, width), generator=gen, device=DEV).to(DT[fmt])
    want = torch.zeros(rows, width, dtype=torch.float64, device=DEV)
    want.index_add_(0, idx[idx >= 0].long(), whole[idx >= 0].double())
    assert torch.equal(wgs.embedding_bwd(whole, idx, rows, 1.0, DT[tfmt]), want.float().to(DT[tfmt]))


@pytest.mark.gpu
def test_sums_keep_the_order_of_positions():
    """A row's terms are added in an order that depends on idx alone: reversing
    which of two equal calls runs first, or what other rows hold, changes no bit
    of it."""
    idx = _indices(30000, 50, "uniform", 5)
    grad = torch.randn(30000, 96, device=DEV)
    first = wgs.embedding_bwd(grad, idx, 50)
    other = torch.where((idx == 7)[:, None], grad, torch.randn_like(grad))
    assert torch.equal(first[7], wgs.embedding_bwd(other, idx, 50)[7])


@pytest.mark.gpu
def test_bad_values_stay_in_their_row_and_column():
    idx = _indices(5000, 40, "uniform", 6)
    grad = torch.randn(5000, 48, device=DEV).half()
    want = wgs.embedding_bwd(grad, idx, 40)
    at = (idx == 7).nonzero()[3].item()
    pad = (idx == -1).nonzero()[0].item()
    grad[at, 5] = float("nan")
    grad[at, 6] = float("inf")
    grad[pad] = float("nan")
    got = wgs.embedding_bwd(grad, idx, 40)
    assert got[7, 5].isnan() and got[7, 6].isinf()
    got[7, 5:7] = want[7, 5:7]
    assert torch.equal(got, want)
    table = torch.randn(40, 48, device=DEV)
    table[7] = float("nan")
    out = wgs.embedding(table, idx)
    assert out[idx == 7].isnan().all() and not out[idx != 7].isnan().any() and (out[pad] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,tfmt", FORMATS)
def test_views_that_start_anywhere(fmt, tfmt):
    n, rows, width = 300, 40, 64
    idx = _indices(n, rows, "skew", 7)
    grad = torch.randn(n, width, device=DEV).to(DT[fmt])
    table = torch.randn(rows, width, device=DEV).to(DT[tfmt])
    for shift in (1, 2, 5):
        gb = torch.full((n * width + 16,), 3.0, dtype=DT[fmt], device=DEV)
        tb = torch.full((rows * width + 16,), 3.0, dtype=DT[tfmt], device=DEV)
        gv, tv = gb[shift:shift + n * width].view(n, width), tb[shift:shift + rows * width].view(rows, width)
        gv.copy_(grad)
        wgs.embedding_bwd(gv, idx, rows, 1.0, DT[tfmt], grad_table=tv)
        _check_gradient(grad, idx, rows, 1.0, tv)
        tv.copy_(table)
        out = wgs.embedding(tv, idx, 2.0, out=gv)
        assert torch.equal(_bits(out), _bits(wgs.embedding(table, idx, 2.0, DT[fmt])))
        for buf, size in ((gb, n * width), (tb, rows * width)):
            assert (buf[:shift] == 3.0).all() and (buf[shift + size:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [100, 5000])
def test_an_index_out_of_range_is_reported_and_takes_no_part(n):
    idx = _indices(n, 30, "uniform", 8)
    grad, table = torch.randn(n, 24, device=DEV), torch.randn(30, 24, device=DEV)
    for bad in (30, -2, 2 ** 31 - 1, -2 ** 31):
        off = idx.clone()
        off[n // 2] = bad
        pad = idx.clone()
        pad[n // 2] = -1
        got = wgs.embedding_bwd(grad, off, 30)
        with pytest.raises(wgs.WgsError, match="WGS_ERR_INDEX"):
            wgs.check_error(DEV)
        assert torch.equal(got, wgs.embedding_bwd(grad, pad, 30))
        out = wgs.embedding(table, off)
        with pytest.raises(wgs.WgsError, match="WGS_ERR_INDEX"):
            wgs.check_error(DEV)
        assert torch.equal(out, wgs.embedding(table, pad))
        wgs.check_error(DEV)


@pytest.mark.gpu
def test_empty_calls_and_python_refusals():
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    table = torch.randn(5, 8, device=DEV)
    assert wgs.embedding(table, none).shape == (0, 8)
    assert (wgs.embedding_bwd(torch.zeros(0, 8, device=DEV), none, 5, grad_table=table.clone()) == 0).all()
    pads = torch.full((6,), -1, dtype=torch.int32, device=DEV)
    assert (wgs.embedding(table[:0], pads) == 0).all()
    assert wgs.embedding_bwd(torch.zeros(6, 8, device=DEV), pads, 0).shape == (0, 8)
    wgs.check_error(DEV)
    idx = torch.tensor([[0, 4, -1], [2, 2, 1]], dtype=torch.int32, device=DEV)
    out = wgs.embedding(table, idx, 0.5)
    assert out.shape == (2, 3, 8) and torch.equal(out[1, 1], table[2] * 0.5)
    grad = wgs.embedding_bwd(out, idx, 5)
    assert torch.equal(grad, wgs.embedding_bwd(out.view(6, 8), idx.view(6), 5))
    assert wgs.embedding(table, idx[0, 0]).shape == (8,)
    for args, kw in (((table, idx.long()), {}), ((table[0], idx), {}), ((table.double(), idx), {}),
                     ((table.half(), idx), {"dtype": torch.bfloat16}), ((table, idx), {"dtype": torch.int32}),
                     ((table, idx), {"out": out[0]}), ((table, idx.t()), {}), ((table.t(), idx), {}),
                     ((table, idx.cpu()), {})):
        with pytest.raises(RuntimeError):
            wgs.embedding(*args, **kw)
    for args, kw in (((out, idx[0], 5), {}), ((out, idx, -1), {}), ((out, idx.long(), 5), {}),
                     ((out.half(), idx, 5), {"dtype": torch.bfloat16}), ((out, idx, 5), {"grad_table": table.half()}),
                     ((out, idx, 5), {"grad_table": table[:4]}), ((out.double(), idx, 5), {}),
                     ((out, idx, 5), {"workspace": torch.zeros(8, dtype=torch.uint8, device=DEV)})):
        with pytest.raises(RuntimeError):
            wgs.embedding_bwd(*args, **kw)
    with pytest.raises(wgs.WgsError, match="WGS_ERR_WIDTH"):
        wgs.embedding(torch.zeros(2, 32769, device=DEV), idx)


@pytest.mark.gpu
@pytest.mark.parametrize("stage", [synth.TINY, synth.TINY_PADDED], ids=lambda s: s.name)
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_the_window_gather_and_its_gradient(stage, fmt):
    """The lookup with scale 1 is window_gather; the gradient through the map is
    the gather by its inverse, and twice that where every row is named twice."""
    idx = wgs.build_window_index(stage.grid, synth.WINDOW, synth.SHIFT, device=DEV)
    inv = wgs.build_window_inverse(stage.grid, synth.WINDOW, synth.SHIFT, device=DEV)
    x = torch.randn(stage.tokens, 192, device=DEV).to(DT[fmt])
    win = wgs.window_gather(x, idx)
    assert torch.equal(_bits(wgs.embedding(x, idx)), _bits(win))
    grad = torch.randn_like(win)
    back = wgs.embedding_bwd(grad, idx, stage.tokens, dtype=DT[fmt])
    assert torch.equal(_bits(back), _bits(wgs.window_gather(grad, inv)))
    twice = wgs.embedding_bwd(torch.cat([grad, grad]), torch.cat([idx, idx]), stage.tokens, dtype=DT[fmt])
    assert torch.equal(_bits(twice), _bits(back + back))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements in a call, looked up and summed: rows of a table
    named in turn, whole numbers."""
    n, rows, width = 3_000_000, 4, 768
    idx = (torch.arange(n, device=DEV) % rows).to(torch.int32)
    table = torch.randint(-4, 5, (rows, width), device=DEV).half()
    out = wgs.embedding(table, idx)
    assert out.numel() > 2 ** 31
    for at in (0, n // 2, n - 4):
        assert torch.equal(out[at:at + 4], table)
    got = wgs.embedding_bwd(out, idx, rows)
    assert torch.equal(got, table.float() * (n // rows))
    del out
    # and a large table
    n, rows, width = 5000, 2_900_000, 768
    idx = _indices(n, rows, "uniform", 9)
    idx[0], idx[1] = rows - 1, 0
    grad = torch.randint(-4, 5, (n, width), device=DEV).half()
    got = wgs.embedding_bwd(grad, idx, rows, 1.0, torch.float16)
    assert got.numel() > 2 ** 31
    want = torch.zeros(n, width, device=DEV)
    named, where = idx[idx >= 0].long().unique(return_inverse=True)
    want.index_add_(0, where, grad[idx >= 0].float())
    assert torch.equal(got[named], want[:named.numel()].half())
    assert torch.equal(wgs.embedding(got, idx)[0], got[rows - 1])
    got[named] = 0
    assert sum(int(got[k:k + 100000].count_nonzero()) for k in range(0, rows, 100000)) == 0


# ---------------------------------------------------------- calls together ----

CALLS = [(180, 366, 192), (9000, 300, 96), (131040, 24, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", CALLS, ids=str)
def test_graph_replay_streams_and_fresh_inputs_give_the_same_bits(shape):
    n, rows, width = shape
    src = [(_indices(n, rows, kind, k), torch.randn(n, width, device=DEV).half(), torch.randn(rows, width, device=DEV))
           for k, kind in enumerate(("uniform", "skew", "once", "one"))]
    idx, grad, table = (t.clone() for t in src[0])

    def run(idx, grad, table):
        return wgs.embedding(table, idx, 1.5, torch.float16), wgs.embedding_bwd(grad, idx, rows, 1.5)

    want = [run(*s) for s in src]
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            captured = run(idx, grad, table)
    torch.cuda.synchronize()
    for _ in range(2):
        for s, ref in zip(src, want):
            with torch.cuda.stream(stream):         # written right before the replay
                for to, value in zip((idx, grad, table), s):
                    to.copy_(value)
                graph.replay()
            eager = [run(*s) for _ in range(2)]     # next to it, on another stream
            torch.cuda.synchronize()
            for got in (captured, *eager):
                assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # written right before eager calls, with nothing between
    got = []
    for s in src * 3:
        for to, value in zip((idx, grad, table), s):
            to.copy_(value)
        got.append(run(idx, grad, table))
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[k % 4]))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", CALLS, ids=str)
def test_calls_with_given_outputs_allocate_nothing(shape):
    n, rows, width = shape
    idx = _indices(n, rows, "uniform", 1)
    grad, table = torch.randn(n, width, device=DEV), torch.randn(rows, width, device=DEV)
    out, got = torch.empty_like(grad), torch.empty_like(table)
    ws = torch.empty(wgs.embedding_bwd_workspace_bytes(n, rows, width), dtype=torch.uint8, device=DEV)

    def calls():
        wgs.embedding(table, idx, out=out)
        wgs.embedding_bwd(grad, idx, rows, grad_table=got, workspace=ws)

    calls()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    allocated, free = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0]
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == allocated
    assert torch.cuda.mem_get_info()[0] == free
