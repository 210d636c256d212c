"""Workloads of the affine layer-norm and embedding operators.

Each case is one call of one operator:

* ``norm``        layer_norm over rows, or residual_add_layer_norm, which adds
                  a branch to the residual stream first;
* ``norm_grad``   layer_norm_bwd: the rows' gradient (with the residual
                  stream's own gradient added where there is one) and the
                  gradients of weight and bias, summed over all rows;
* ``embed``       embedding: rows of a table by index, scaled;
* ``embed_grad``  embedding_bwd: the table's gradient, the gradients of all
                  outputs summed by index.

With ``own`` false the operators are computed in elementary torch operations;
with ``own`` true by this repository's package.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # the cells of one 2 x 6 x 12 window: next to no work, the call's
        # latency is what counts
        {"name": "norm_window", "op": "norm", "rows": 144, "width": 192, "residual": False,
         "weight": True, "dtype": "bf16", "param": "f32"},
        # every token of the 192-channel stage
        {"name": "norm_192", "op": "norm", "rows": 131040, "width": 192, "residual": False,
         "weight": True, "dtype": "f16", "param": "f32"},
        # a residual stream of odd width with a class row in front of the
        # 384-channel stage's tokens: no row but the first starts on 16 bytes
        {"name": "norm_residual_odd", "op": "norm", "rows": 32761, "width": 771, "residual": True,
         "weight": True, "dtype": "bf16", "param": "bf16"},
        # training on a single window
        {"name": "norm_grad_window", "op": "norm_grad", "rows": 144, "width": 192,
         "residual": False, "weight": True, "dtype": "f32", "param": "f32"},
        # training the 192-channel stage
        {"name": "norm_grad_192", "op": "norm_grad", "rows": 131040, "width": 192,
         "residual": False, "weight": True, "dtype": "f16", "param": "f32"},
        # a wide residual stream, as wide as the 384-channel stage's hidden layer
        {"name": "norm_grad_residual_1536", "op": "norm_grad", "rows": 32760, "width": 1536,
         "residual": True, "weight": True, "dtype": "bf16", "param": "bf16"},
        # the codes of one latitude row looked up in a table of days
        {"name": "embed_row", "op": "embed", "n": 180, "table_rows": 366, "width": 192,
         "kind": "uniform", "pad": 0.0, "table": "f32", "dtype": "bf16"},
        # a batch of long token sequences, a few words making up most of it
        {"name": "embed_tokens", "op": "embed", "n": 131040, "table_rows": 32768, "width": 384,
         "kind": "zipf", "pad": 0.05, "table": "f32", "dtype": "bf16"},
        # training the table of days on one latitude row
        {"name": "embed_grad_row", "op": "embed_grad", "n": 180, "table_rows": 366, "width": 192,
         "kind": "uniform", "pad": 0.0, "table": "f32", "dtype": "f32"},
        # 24 surface classes over the whole grid: thousands of tokens a row
        {"name": "embed_grad_classes", "op": "embed_grad", "n": 131040, "table_rows": 24,
         "width": 192, "kind": "uniform", "pad": 0.0, "table": "f32", "dtype": "f16"},
        # training the table of long token sequences
        {"name": "embed_grad_tokens", "op": "embed_grad", "n": 131040, "table_rows": 32768,
         "width": 384, "kind": "zipf", "pad": 0.05, "table": "f32", "dtype": "bf16"},
        # the way back through the shifted windows of the 192-channel stage:
        # every token named once, the windows' pads by nobody
        {"name": "embed_grad_windows", "op": "embed_grad", "kind": "windows", "gz": 8, "gh": 91,
         "gw": 180, "width": 192, "table": "f16", "dtype": "f16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "embed", "embed_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    param = rng.choice(["f32", dtype])
    if op in ("norm", "norm_grad"):
        # a row of a handful of values has no statistics to speak of
        width = _log_int(rng, 16, 8192)
        if rng.random() < 0.4:
            width = -(-width // 64) * 64
        # at most the work of the largest listed case of the same operator
        most = 32761 * 771 if op == "norm" else 32760 * 1536
        if dtype == "f32":
            most //= 2
        rows = _log_int(rng, 1, max(1, min(131040, most // width)))
        return {"op": op, "rows": rows, "width": width, "residual": rng.random() < 0.4,
                "weight": rng.random() < 0.85, "dtype": dtype, "param": param}
    width = _log_int(rng, 1, 2048)
    if rng.random() < 0.4:
        width = -(-width // 64) * 64
    most = 131040 * 384
    if dtype == "f32":
        most //= 2
    if rng.random() < 0.2:
        grid = [rng.randint(1, 8), rng.randint(1, 91), rng.randint(1, 180)]
        while -(-grid[0] // 2) * 2 * -(-grid[1] // 6) * 6 * -(-grid[2] // 12) * 12 * width > most // 2:
            grid[grid.index(max(grid))] //= 2
        return {"op": op, "kind": "windows", "gz": grid[0], "gh": grid[1], "gw": grid[2],
                "width": width, "table": param, "dtype": dtype}
    n = _log_int(rng, 1, min(131040, most // width))
    table_rows = _log_int(rng, 1, min(262144, 32768 * 384 // width))
    return {"op": op, "n": n, "table_rows": table_rows, "width": width,
            "kind": rng.choice(["zipf", "uniform"]), "pad": rng.choice([0.0, 0.05, 0.5]),
            "table": param, "dtype": dtype}


# ------------------------------------------------------------------ state ----

def _window_map(grid):
    """int64 on the host: the token of every row of the grid's 2 x 6 x 12
    windows, rolled by half a window, -1 for a row past the grid's end."""
    win, shift = (2, 6, 12), (1, 3, 6)
    padded = [-(-g // w) * w for g, w in zip(grid, win)]
    tokens = torch.arange(grid[0] * grid[1] * grid[2]).reshape(grid)
    tokens = torch.roll(tokens, [-s for s in shift], (0, 1, 2))
    full = torch.full(padded, -1, dtype=torch.int64)
    full[:grid[0], :grid[1], :grid[2]] = tokens
    (z, wz), (h, wh), (w, ww) = ((p // k, k) for p, k in zip(padded, win))
    return full.reshape(z, wz, h, wh, w, ww).permute(0, 2, 4, 1, 3, 5).reshape(-1)


def _sizes(case):
    """(indices, rows of the table) of an embedding case."""
    if case["kind"] == "windows":
        g = case["gz"], case["gh"], case["gw"]
        return (-(-g[0] // 2) * 2 * -(-g[1] // 6) * 6 * -(-g[2] // 12) * 12, g[0] * g[1] * g[2])
    return case["n"], case["table_rows"]


def _indices(case, gen):
    if case["kind"] == "windows":
        return _window_map((case["gz"], case["gh"], case["gw"])).to(torch.int32).cuda()
    n, rows = case["n"], case["table_rows"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if case["kind"] == "zipf":      # the k-th most frequent in proportion to 1 / k
        rank = torch.exp(u * math.log(rows + 1)).long() - 1
        place = torch.randperm(rows, generator=gen, device="cuda")
        idx = place[rank.clamp(0, rows - 1)]
    else:
        idx = (u * rows).long().clamp(max=rows - 1)
    if case["pad"] > 0:             # positions behind the sequences' ends
        gone = torch.rand(n, generator=gen, device="cuda") < case["pad"]
        idx = torch.where(gone, -1, idx)
    return idx.to(torch.int32)


def _randn(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] in ("embed", "embed_grad"):
        n, rows = _sizes(case)
        st["idx"] = _indices(case, gen)
        # a factor that 32 bits hold
        st["scale"] = torch.tensor(math.sqrt(case["width"]), dtype=torch.float32).item()
        if case["op"] == "embed":
            st["table"] = _randn(gen, (rows, case["width"]), 0.02).to(_DTYPES[case["table"]])
            return st
        st["grad"] = _randn(gen, (n, case["width"]), 0.05).to(dt)
        if own:
            import window_gather_swin_gb300 as wgs
            st["workspace"] = torch.empty(
                wgs.embedding_bwd_workspace_bytes(n, rows, case["width"]), dtype=torch.uint8,
                device="cuda")
        return st
    rows, width = case["rows"], case["width"]
    pt = _DTYPES[case["param"]]
    # channels with scales and offsets of their own, as blocks leave them
    scale = 0.5 + torch.rand(width, generator=gen, device="cuda")
    st["x"] = (_randn(gen, (rows, width)) * scale + _randn(gen, (width,))).to(dt)
    st["weight"] = st["bias"] = None
    if case["weight"]:
        st["weight"] = (1.0 + _randn(gen, (width,), 0.2)).to(pt)
        st["bias"] = _randn(gen, (width,), 0.2).to(pt)
    if case["op"] == "norm":
        if case["residual"]:
            st["branch"] = _randn(gen, (rows, width), 0.5).to(dt)
        return st
    st["grad"] = _randn(gen, (rows, width), 0.1).to(dt)
    if case["residual"]:
        st["grad_residual"] = _randn(gen, (rows, width), 0.1).to(dt)
    # what the forward pass left: every row's statistics
    mean = st["x"].double().mean(1)
    var = (st["x"].double() - mean[:, None]).square().mean(1)
    st["mean"], st["rstd"] = mean.float(), (var + EPS).rsqrt().float()
    if own:
        import window_gather_swin_gb300 as wgs
        st["workspace"] = torch.empty(wgs.layer_norm_bwd_workspace_bytes(rows, width),
                                      dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- plain forms ----

def _plain_norm(st):
    c, x = st["case"], st["x"]
    total = None
    if c["residual"]:
        # the residual stream is kept in the tensors' format, and the norm
        # starts from what is kept
        total = x = (x.float() + st["branch"].float()).to(x.dtype)
    xf = x.float()
    mean = xf.sum(1) / c["width"]
    d = xf - mean[:, None]
    var = (d * d).sum(1) / c["width"]
    rstd = 1.0 / torch.sqrt(var + EPS)
    y = d * rstd[:, None]
    if c["weight"]:
        y = y * st["weight"].float() + st["bias"].float()
    y = y.to(x.dtype)
    return (total, y, mean, rstd) if c["residual"] else (y, mean, rstd)


def _plain_norm_grad(st):
    c = st["case"]
    g = st["grad"].float()
    h = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    grad_w = grad_b = None
    if c["weight"]:
        grad_w = (g * h).sum(0, dtype=torch.float64).to(st["weight"].dtype)
        grad_b = g.sum(0, dtype=torch.float64).to(st["bias"].dtype)
        g = g * st["weight"].float()
    m1 = g.sum(1, keepdim=True) / c["width"]
    m2 = (g * h).sum(1, keepdim=True) / c["width"]
    grad_x = (g - m1 - h * m2) * st["rstd"][:, None]
    if c["residual"]:
        grad_x = grad_x + st["grad_residual"].float()
    return grad_x.to(st["x"].dtype), grad_w, grad_b


def _plain_embed(st):
    idx = st["idx"].long()
    out = st["table"].float()[idx.clamp(min=0)] * st["scale"]
    return torch.where((idx >= 0)[:, None], out, 0.0).to(_DTYPES[st["case"]["dtype"]])


def _plain_embed_grad(st):
    c = st["case"]
    rows = _sizes(c)[1]
    idx = st["idx"].long()
    idx = torch.where(idx >= 0, idx, rows)                # a last row takes the rest
    total = torch.zeros(rows + 1, c["width"], dtype=torch.float64, device="cuda")
    total.index_add_(0, idx, st["grad"].double())
    return (total[:rows] * st["scale"]).to(_DTYPES[c["table"]])


def run(state):
    c = state["case"]
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "embed": _plain_embed,
                "embed_grad": _plain_embed_grad}[c["op"]](state)
    import window_gather_swin_gb300 as wgs
    if c["op"] == "norm":
        if c["residual"]:
            return wgs.residual_add_layer_norm(state["x"], state["branch"], state["weight"],
                                               state["bias"], EPS)
        return wgs.layer_norm(state["x"], state["weight"], state["bias"], EPS)
    if c["op"] == "norm_grad":
        return wgs.layer_norm_bwd(state["grad"], state["x"], state["mean"], state["rstd"],
                                  state["weight"], state.get("grad_residual"),
                                  workspace=state["workspace"])
    if c["op"] == "embed":
        return wgs.embedding(state["table"], state["idx"], state["scale"],
                             dtype=_DTYPES[c["dtype"]])
    return wgs.embedding_bwd(state["grad"], state["idx"], _sizes(c)[1], state["scale"],
                             dtype=_DTYPES[c["table"]], workspace=state["workspace"])


# -------------------------------------------------------------------- work ----

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    if case["op"] in ("embed", "embed_grad"):
        n, rows = _sizes(case)
        width = case["width"]
        if case["op"] == "embed_grad":
            # the sums of all rows' gradients, and every row of the table written
            return {"bytes": n * (4 + width * _size(case["dtype"])) + rows * width * _size(case["table"]),
                    "flops": (n + rows) * width}
        # rows that are named are read once, however often they are named
        if case["kind"] == "windows":
            named = rows
        elif case["kind"] == "uniform":
            named = rows * -math.expm1(n * (1 - case["pad"]) * math.log1p(-1 / max(rows, 2)))
        else:
            total = math.log(rows + 1)
            named = sum(-math.expm1(-n * (1 - case["pad"]) * math.log1p(1 / k) / total)
                        for k in range(1, rows + 1))
        named = max(1, min(n, rows, round(named)))
        return {"bytes": n * (4 + width * _size(case["dtype"])) + named * width * _size(case["table"]),
                "flops": n * width}
    items, rows = case["rows"] * case["width"], case["rows"]
    params = 2 * case["width"] * _size(case["param"]) if case["weight"] else 0
    tensors = 2 if case["op"] == "norm" else 3
    if case["residual"]:
        tensors += 2 if case["op"] == "norm" else 1
    stats = 8 * rows
    if case["op"] == "norm":
        # a sum, a difference, its square and its sum, and the scale; weight and bias
        per = 5 + (2 if case["weight"] else 0) + (1 if case["residual"] else 0)
        return {"bytes": tensors * items * _size(case["dtype"]) + params + stats,
                "flops": items * per}
    per = 10 + (4 if case["weight"] else 0) + (1 if case["residual"] else 0)
    # weight is read, the gradients of weight and bias are written
    return {"bytes": tensors * items * _size(case["dtype"]) + params * 3 // 2 + stats,
            "flops": items * per}


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "embed":
        held = st["idx"] >= 0
        out = torch.zeros(held.numel(), case["width"], dtype=torch.float64, device="cuda")
        out[held] = st["table"].double()[st["idx"][held].long()] * st["scale"]
        return out
    if case["op"] == "embed_grad":
        # the tokens in the order of their indices:
        # every row's own tokens are added up
        rows, width = _sizes(case)[1], case["width"]
        order = torch.argsort(st["idx"], stable=True)
        order = order[st["idx"][order] >= 0]
        counts = torch.bincount(st["idx"][order].long(), minlength=rows)
        if order.numel() == 0:
            return torch.zeros(rows, width, dtype=torch.float64, device="cuda")
        out = torch.empty(rows, width, dtype=torch.float64, device="cuda")
        for lo in range(0, width, 64):
            part = st["grad"][order, lo:lo + 64].double()
            out[:, lo:lo + 64] = torch.segment_reduce(part, "sum", lengths=counts, axis=0, initial=0)
        return out * st["scale"]
    x = st["x"].double()
    w = st["weight"].double() if case["weight"] else torch.ones(case["width"], device="cuda").double()
    if case["op"] == "norm":
        total = None
        if case["residual"]:
            total = x = (x + st["branch"].double()).to(_DTYPES[case["dtype"]]).double()
        mean = x.mean(1, keepdim=True)
        rstd = (x.var(1, unbiased=False, keepdim=True) + EPS) ** -0.5
        y = (x - mean) * rstd * w
        if case["weight"]:
            y = y + st["bias"].double()
        out = (y, mean[:, 0], rstd[:, 0])
        return (total, *out) if case["residual"] else out
    rstd = st["rstd"].double()[:, None]
    h = (x - st["mean"].double()[:, None]) * rstd
    g = st["grad"].double()
    gw = gb = None
    if case["weight"]:
        gb = g.sum(0)
        gw = torch.einsum("ij,ij->j", g, h)
    g = g * w
    gx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    if case["residual"]:
        gx = gx + st["grad_residual"].double()
    return gx, gw, gb
