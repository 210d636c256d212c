"""Workloads of the position-bias and group-norm operators.

Each case is one call of one operator:

* ``bias``       position_bias: the attention bias of every window type and
                 head, expanded from a learned table by a bucket map;
* ``bias_grad``  position_bias_bwd: the table's gradient, from the gradient of
                 the logits of every window;
* ``norm``       group_norm_act: group norm over channels-last rows with the
                 activation behind it;
* ``norm_grad``  group_norm_act_bwd: its gradients.

With ``own`` false the operators are computed in elementary torch operations;
with ``own`` true by this repository's package.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ----

def listed():
    win = {"map": "window", "wz": 2, "wh": 6, "ww": 12}
    return [
        # one type's bias for the attention of a 6-head block, laid out before
        # every training step: little work, the call's latency is what counts
        {"name": "bias_window", "op": "bias", **win, "absolute": 0, "types": 1, "heads": 6,
         "table": "f32", "dtype": "bf16"},
        # the 192-channel stage: 64 latitude bands with tables of their own,
        # depth and latitude absolute, longitude relative
        {"name": "bias_window_types", "op": "bias", **win, "absolute": 3, "types": 64, "heads": 6,
         "table": "f32", "dtype": "f16"},
        # logarithmic distance buckets over a long sequence of odd length
        {"name": "bias_distance", "op": "bias", "map": "distance", "nq": 2047, "nk": 2047,
         "buckets": 32, "reach": 128, "both": True, "types": 1, "heads": 16,
         "table": "bf16", "dtype": "bf16"},
        # the gradient of the 192-channel stage's tables, from 960 windows
        {"name": "bias_grad_types", "op": "bias_grad", **win, "absolute": 3, "types": 64,
         "heads": 6, "windows": 960, "order": "runs", "table": "f32", "dtype": "f16"},
        # the 384-channel stage with one table shared by its 256 windows
        {"name": "bias_grad_shared", "op": "bias_grad", **win, "absolute": 0, "types": 1,
         "heads": 12, "windows": 256, "order": "none", "table": "bf16", "dtype": "bf16"},
        # flat 7 x 7 windows: 49 x 49 logits, so no tile starts on 16 bytes
        {"name": "bias_grad_odd", "op": "bias_grad", "map": "window", "wz": 1, "wh": 7, "ww": 7,
         "absolute": 0, "types": 1, "heads": 12, "windows": 1024, "order": "none",
         "table": "f32", "dtype": "f16"},
        # causal distance buckets: long rows, half of the pairs hold no bucket
        {"name": "bias_grad_distance", "op": "bias_grad", "map": "distance", "nq": 1024,
         "nk": 1024, "buckets": 32, "reach": 128, "both": False, "types": 1, "heads": 8,
         "windows": 2, "order": "none", "table": "f32", "dtype": "f32"},
        # a small level of a sampling path, odd in every extent
        {"name": "norm_small", "op": "norm", "n": 2, "spatial": 143, "channels": 90, "groups": 6,
         "act": "silu", "dtype": "f32", "param": "f32"},
        # the whole 192-channel token grid of one sample
        {"name": "norm_192", "op": "norm", "n": 1, "spatial": 131040, "channels": 192,
         "groups": 32, "act": "silu", "dtype": "f16", "param": "f32"},
        # a batch of 384-channel grids, larger than the chip's cache
        {"name": "norm_384_batch", "op": "norm", "n": 8, "spatial": 32760, "channels": 384,
         "groups": 32, "act": "gelu_tanh", "dtype": "bf16", "param": "bf16"},
        # training the 192-channel level
        {"name": "norm_grad_192", "op": "norm_grad", "n": 1, "spatial": 131040, "channels": 192,
         "groups": 32, "act": "silu", "dtype": "f16", "param": "f32"},
        # training the 384-channel level with a batch
        {"name": "norm_grad_384_batch", "op": "norm_grad", "n": 4, "spatial": 32760,
         "channels": 384, "groups": 32, "act": "gelu_tanh", "dtype": "bf16", "param": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_map(rng, most):
    """A bucket map of at most `most` pairs."""
    if rng.random() < 0.6:
        while True:
            c = {"map": "window", "wz": rng.randint(1, 3), "wh": rng.randint(1, 12),
                 "ww": rng.randint(1, 12), "absolute": rng.randint(0, 7)}
            if (c["wz"] * c["wh"] * c["ww"]) ** 2 <= most:
                return c
    nk = _log_int(rng, 1, 2047)
    nq = 1 if rng.random() < 0.25 else _log_int(rng, 1, min(2047, max(1, most // nk)))
    return {"map": "distance", "nq": nq, "nk": nk, "buckets": 2 * rng.randint(2, 32),
            "reach": _log_int(rng, 40, 1024), "both": rng.random() < 0.5}


def draw(rng):
    op = rng.choice(["bias", "bias_grad", "norm", "norm_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    param = rng.choice(["f32", dtype])
    if op in ("bias", "bias_grad"):
        # at most the work of the largest listed case of the same operator
        most = 2047 * 2047 * 16 if op == "bias" else 960 * 6 * 144 * 144
        if dtype == "f32":
            most //= 2
        c = {"op": op, **_draw_map(rng, min(most, 2047 * 2047)), "table": param, "dtype": dtype}
        np_ = _pairs(c)[0] * _pairs(c)[1]
        c["heads"] = _log_int(rng, 1, max(1, min(32, most // np_)))
        if op == "bias":
            c["types"] = _log_int(rng, 1, max(1, min(64, most // (np_ * c["heads"]))))
            # tables stay of a realistic size beside the bias they give
            while c["types"] > 1 and c["types"] * _buckets(c) * c["heads"] > 4 << 20:
                c["types"] //= 2
            return c
        c["windows"] = _log_int(rng, 1, max(1, min(4096, most // (np_ * c["heads"]))))
        c["order"] = rng.choice(["none", "runs", "mixed"])
        c["types"] = 1 if c["order"] == "none" else _log_int(rng, 1, max(1, min(64, c["windows"])))
        while c["types"] > 1 and c["types"] * _buckets(c) * c["heads"] > 4 << 20:
            c["types"] //= 2
        return c
    groups = rng.choice([1, 2, 3, 4, 6, 8, 16, 32])
    per = _log_int(rng, 1, max(1, 1024 // groups))
    channels = groups * per
    most = (8 if op == "norm" else 4) * 32760 * 384
    if dtype == "f32":
        most //= 2
    n = _log_int(rng, 1, 16)
    # a group of a handful of values has no statistics to speak of
    least = -(-64 // per)
    spatial = _log_int(rng, least, max(least, min(131040, most // (n * channels))))
    return {"op": op, "n": n, "spatial": spatial, "channels": channels, "groups": groups,
            "act": rng.choice(["none", "silu", "gelu_tanh"]), "dtype": dtype, "param": param}


# ------------------------------------------------------------------- maps ----

def _pairs(case):
    if case["map"] == "window":
        n = case["wz"] * case["wh"] * case["ww"]
        return n, n
    return case["nq"], case["nk"]


def _buckets(case):
    if case["map"] == "distance":
        return case["buckets"]
    total = 1
    for axis, w in enumerate((case["wz"], case["wh"], case["ww"])):
        total *= w * w if case["absolute"] >> axis & 1 else 2 * w - 1
    return total


def _bucket_map(case):
    """int32 [nq, nk] on the host: the table row of every (query, key) pair,
    -1 for a pair without one."""
    if case["map"] == "window":
        ext = (case["wz"], case["wh"], case["ww"])
        cells = torch.stack(torch.meshgrid(*(torch.arange(w) for w in ext), indexing="ij"))
        cells = cells.reshape(3, -1)
        out = torch.zeros(cells.shape[1], cells.shape[1], dtype=torch.int64)
        for axis, w in enumerate(ext):
            a, b = cells[axis][:, None], cells[axis][None, :]
            if case["absolute"] >> axis & 1:
                out = out * (w * w) + a * w + b
            else:
                out = out * (2 * w - 1) + a - b + w - 1
        return out.to(torch.int32)
    nq, nk, both = case["nq"], case["nk"], case["both"]
    start = nk - nq if nk > nq else 0      # the queries are the last positions
    d = torch.arange(nk)[None, :] - (torch.arange(nq)[:, None] + start)     # key - query
    buckets = case["buckets"]
    half = buckets // 2 if both else buckets
    exact_n = half // 2
    away = d.abs() if both else (-d).clamp(min=0)
    far = (away.clamp(min=1).double() / exact_n).log() / math.log(case["reach"] / exact_n)
    far = exact_n + (far * (half - exact_n) + 1e-9).floor().long()
    out = torch.where(away < exact_n, away, far.clamp(max=half - 1))
    if both:
        out = out + half * (d > 0)
    else:
        out = torch.where(d > 0, -1, out)
    return out.to(torch.int32)


# ------------------------------------------------------------------ state ----

def _randn(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] in ("bias", "bias_grad"):
        nq, nk = _pairs(case)
        bucket = _bucket_map(case)
        st["buckets"] = _buckets(case)
        if case["op"] == "bias":
            st["bucket"] = bucket.cuda()
            st["table"] = _randn(gen, (case["types"], st["buckets"], case["heads"]), 0.02).to(
                _DTYPES[case["table"]])
            return st
        w = case["windows"]
        st["grad"] = torch.empty(w, case["heads"], nq, nk, dtype=dt, device="cuda")
        for i in range(0, w, 64):          # gradients of logits, loss-scaled
            part = st["grad"][i:i + 64]
            part.copy_(_randn(gen, part.shape, 0.05))
        st["type"] = None
        if case["order"] == "runs":        # the windows of a band follow one another
            st["type"] = (torch.arange(w, device="cuda") * case["types"] // w).to(torch.int32)
        elif case["order"] == "mixed":
            st["type"] = torch.randint(0, case["types"], (w,), generator=gen, device="cuda",
                                       dtype=torch.int32)
        if own:
            import window_gather_swin_gb300 as wgs
            st["plan"] = wgs.build_bucket_plan(bucket, st["buckets"], device="cuda")
            st["workspace"] = torch.empty(
                wgs.position_bias_bwd_workspace_bytes(st["plan"], w, case["heads"], case["types"]),
                dtype=torch.uint8, device="cuda")
        st["bucket"] = bucket.cuda()
        return st
    n, s, c, g = case["n"], case["spatial"], case["channels"], case["groups"]
    pt = _DTYPES[case["param"]]
    # channels with scales and offsets of their own, as a convolution leaves them
    scale = 0.5 + torch.rand(c, generator=gen, device="cuda")
    offset = _randn(gen, (c,), 1.0)
    st["x"] = torch.empty(n, s, c, dtype=dt, device="cuda")
    for i in range(n):
        st["x"][i].copy_(_randn(gen, (s, c)) * scale + offset)
    st["weight"] = (1.0 + _randn(gen, (c,), 0.2)).to(pt)
    st["bias"] = _randn(gen, (c,), 0.2).to(pt)
    if case["op"] == "norm_grad":
        st["grad"] = torch.empty(n, s, c, dtype=dt, device="cuda")
        for i in range(n):
            st["grad"][i].copy_(_randn(gen, (s, c), 0.1))
        # what the forward pass left: statistics of every sample and group
        x = st["x"].view(n, s, g, c // g)
        mean = x.double().mean((1, 3))
        var = (x.double() - mean[:, None, :, None]).square().mean((1, 3))
        st["mean"], st["rstd"] = mean.float(), (var + 1e-5).rsqrt().float()
    if own:
        import window_gather_swin_gb300 as wgs
        need = (wgs.group_norm_act_workspace_bytes if case["op"] == "norm"
                else wgs.group_norm_act_bwd_workspace_bytes)
        st["workspace"] = torch.empty(need(n, s, c, g), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- plain forms ----

def _plain_bias(st):
    c = st["case"]
    nq, nk = _pairs(c)
    idx = st["bucket"].view(-1).long()
    out = st["table"].float()[:, idx.clamp(min=0)]                   # [types, pairs, heads]
    out = torch.where(idx[None, :, None] >= 0, out, 0.0)
    out = out.permute(0, 2, 1).to(_DTYPES[c["dtype"]])
    return out.reshape(c["types"], c["heads"], nq, nk)


def _plain_bias_grad(st):
    c = st["case"]
    nq, nk = _pairs(c)
    grad = st["grad"].view(c["windows"], c["heads"], nq * nk)
    if st["type"] is None:
        per_type = grad.sum(0, keepdim=True, dtype=torch.float64)
    else:
        per_type = torch.zeros(c["types"], c["heads"], nq * nk, dtype=torch.float64, device="cuda")
        per_type.index_add_(0, st["type"].long(), grad.double())
    idx = st["bucket"].view(-1).long()
    idx = torch.where(idx >= 0, idx, st["buckets"])                  # a last row takes the rest
    table = torch.zeros(c["types"], c["heads"], st["buckets"] + 1, dtype=torch.float64,
                        device="cuda")
    table.index_add_(2, idx, per_type)
    return table[:, :, :-1].permute(0, 2, 1).contiguous().to(_DTYPES[c["table"]])


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-2.0 * k * (z + 0.044715 * z * z * z)))
        return s + z * s * (1.0 - s) * 2.0 * k * (1.0 + 3.0 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_norm(st):
    c = st["case"]
    n, s, ch, g = c["n"], c["spatial"], c["channels"], c["groups"]
    x = st["x"].float().view(n, s, g, ch // g)
    count = s * (ch // g)
    mean = (x.sum((1, 3), dtype=torch.float64) / count).float()
    xc = x - mean[:, None, :, None]
    var = (xc * xc).sum((1, 3), dtype=torch.float64) / count
    rstd = (1.0 / torch.sqrt(var + 1e-5)).float()
    z = (xc * rstd[:, None, :, None]).view(n, s, ch) * st["weight"].float() + st["bias"].float()
    return _act(z, c["act"]).to(st["x"].dtype), mean, rstd


def _plain_norm_grad(st):
    c = st["case"]
    n, s, ch, g = c["n"], c["spatial"], c["channels"], c["groups"]
    w, b = st["weight"].float(), st["bias"].float()
    xh = (st["x"].float().view(n, s, g, ch // g) - st["mean"][:, None, :, None])
    xh = (xh * st["rstd"][:, None, :, None]).view(n, s, ch)
    dz = st["grad"].float() * _act_grad(xh * w + b, c["act"])
    grad_b = dz.sum((0, 1), dtype=torch.float64)
    grad_w = (dz * xh).sum((0, 1), dtype=torch.float64)
    dxh = (dz * w).view(n, s, g, ch // g)
    xg = xh.view(n, s, g, ch // g)
    count = s * (ch // g)
    m1 = (dxh.sum((1, 3), dtype=torch.float64) / count).float()[:, None, :, None]
    m2 = ((dxh * xg).sum((1, 3), dtype=torch.float64) / count).float()[:, None, :, None]
    grad_x = (dxh - m1 - xg * m2) * st["rstd"][:, None, :, None]
    return (grad_x.view(n, s, ch).to(st["x"].dtype), grad_w.to(st["weight"].dtype),
            grad_b.to(st["bias"].dtype))


def run(state):
    c = state["case"]
    if not own:
        return {"bias": _plain_bias, "bias_grad": _plain_bias_grad, "norm": _plain_norm,
                "norm_grad": _plain_norm_grad}[c["op"]](state)
    import window_gather_swin_gb300 as wgs
    if c["op"] == "bias":
        return wgs.position_bias(state["table"], state["bucket"], dtype=_DTYPES[c["dtype"]])
    if c["op"] == "bias_grad":
        return wgs.position_bias_bwd(state["grad"], state["plan"], state["type"], c["types"],
                                     dtype=_DTYPES[c["table"]], workspace=state["workspace"])
    if c["op"] == "norm":
        return wgs.group_norm_act(state["x"], c["groups"], state["weight"], state["bias"], 1e-5,
                                  c["act"], workspace=state["workspace"])
    return wgs.group_norm_act_bwd(state["grad"], state["x"], c["groups"], state["mean"],
                                  state["rstd"], state["weight"], state["bias"], c["act"],
                                  workspace=state["workspace"])


# -------------------------------------------------------------------- work ----

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    if case["op"] in ("bias", "bias_grad"):
        nq, nk = _pairs(case)
        table = case["types"] * _buckets(case) * case["heads"] * _size(case["table"])
        if case["op"] == "bias":
            out = case["types"] * case["heads"] * nq * nk
            return {"bytes": table + 4 * nq * nk + out * _size(case["dtype"]), "flops": 0}
        grad = case["windows"] * case["heads"] * nq * nk
        kinds = 0 if case["order"] == "none" else 4 * case["windows"]
        return {"bytes": table + 4 * nq * nk + kinds + grad * _size(case["dtype"]), "flops": grad}
    n, s, ch, g = case["n"], case["spatial"], case["channels"], case["groups"]
    items = n * s * ch
    stats = 2 * 4 * n * g
    act = {"none": 0, "silu": 4, "gelu_tanh": 9}[case["act"]]
    if case["op"] == "norm":
        # two for the mean and four for the variance and the norm, then scale and shift
        return {"bytes": 2 * items * _size(case["dtype"]) + 2 * ch * _size(case["param"]) + stats,
                "flops": items * (8 + act)}
    return {"bytes": 3 * items * _size(case["dtype"]) + 4 * ch * _size(case["param"]) + stats,
            "flops": items * (16 + 2 * act)}


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "bias":
        nq, nk = _pairs(case)
        table = st["table"].double()
        idx = st["bucket"].long()
        out = torch.zeros(case["types"], case["heads"], nq, nk, dtype=torch.float64, device="cuda")
        held = idx >= 0
        for t in range(case["types"]):
            for h in range(case["heads"]):
                out[t, h][held] = table[t, :, h][idx[held]]
        return out
    if case["op"] == "bias_grad":
        idx = st["bucket"].view(-1).long()
        held = idx >= 0
        out = torch.zeros(case["types"], st["buckets"], case["heads"], dtype=torch.float64,
                          device="cuda")
        for t in range(case["types"]):
            if st["type"] is None:
                mine = range(case["windows"])
            else:
                mine = (st["type"] == t).nonzero().view(-1).tolist()
            for h in range(case["heads"]):
                total = torch.zeros(idx.numel(), dtype=torch.float64, device="cuda")
                for part in range(0, len(mine), 64):
                    sel = torch.tensor(mine[part:part + 64], device="cuda")
                    total += st["grad"][sel, h].reshape(len(sel), -1).double().sum(0)
                if bool(held.any()):
                    out[t, :, h] = torch.bincount(idx[held], total[held], minlength=st["buckets"])
        return out
    n, ch, g = case["n"], case["channels"], case["groups"]
    cols = ch // g
    w, b = st["weight"].double(), st["bias"].double()
    y = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")      # or grad_x
    if case["op"] == "norm":
        mean = torch.empty(n, g, dtype=torch.float64, device="cuda")
        rstd = torch.empty(n, g, dtype=torch.float64, device="cuda")
    else:
        gw = torch.zeros(ch, dtype=torch.float64, device="cuda")
        gb = torch.zeros_like(gw)
    k = math.sqrt(2.0 / math.pi)
    for i in range(n):
        for j in range(g):
            at = slice(j * cols, (j + 1) * cols)
            x = st["x"][i, :, at].double()
            if case["op"] == "norm":
                mean[i, j] = x.mean()
                rstd[i, j] = (x.var(unbiased=False) + 1e-5) ** -0.5
                r, m = rstd[i, j], mean[i, j]
            else:
                r, m = st["rstd"][i, j].double(), st["mean"][i, j].double()
            xh = (x - m) * r
            z = xh * w[at] + b[at]
            u = k * (z + 0.044715 * z ** 3)
            half = torch.sigmoid(z if case["act"] == "silu" else 2.0 * u)
            if case["op"] == "norm":
                y[i, :, at] = z if case["act"] == "none" else z * half
                continue
            if case["act"] == "none":
                slope = torch.ones_like(z)
            else:
                du = 1.0 if case["act"] == "silu" else 2.0 * k * (1.0 + 3.0 * 0.044715 * z * z)
                slope = half + z * half * torch.sigmoid(-(z if case["act"] == "silu" else 2.0 * u)) * du
            dz = st["grad"][i, :, at].double() * slope
            gb[at] += dz.sum(0)
            gw[at] += (dz * xh).sum(0)
            d = dz * w[at]
            y[i, :, at] = r * (d - d.mean() - xh * (d * xh).mean())
    return (y, mean, rstd) if case["op"] == "norm" else (y, gw, gb)
