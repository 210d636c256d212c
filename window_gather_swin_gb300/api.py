"""Python entry points, one per C-ABI function, with the same names.

Each function checks what the C ABI cannot see (device, dtype, contiguity,
shapes of torch tensors), allocates outputs the caller did not pass, and
hands raw pointers plus the current CUDA stream of the tensors' device to
libwgs.so.  No arithmetic of the op happens here, and there is no CPU path:
CPU tensors are rejected.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import _capi

_DTYPE = {torch.float32: _capi.WGS_F32, torch.float16: _capi.WGS_F16,
          torch.bfloat16: _capi.WGS_BF16}
LN_WIDTHS = (192, 384)
ROW_DTYPES = (torch.float16, torch.bfloat16)


def _entry(name: str, dtype):
    """The C entry point for a 16-bit row op: fp16 `name`, bfloat16 `name_bf16`."""
    return getattr(_capi.load(), name if dtype == torch.float16 else name + "_bf16")


def _row16(t: torch.Tensor, name: str) -> None:
    _cuda(t, name)
    _require(t.dtype in ROW_DTYPES, f"{name} must be float16 or bfloat16 (got {t.dtype})")


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise RuntimeError(msg)


def _cuda(t: torch.Tensor, name: str, dtype=None) -> None:
    _require(isinstance(t, torch.Tensor), f"{name} must be a torch.Tensor")
    _require(t.is_cuda, f"{name} must be a CUDA tensor (got {t.device})")
    if dtype is not None:
        _require(t.dtype == dtype, f"{name} must be {dtype} (got {t.dtype})")
    _require(t.is_contiguous(), f"{name} must be contiguous")


def _same_device(*ts: torch.Tensor) -> None:
    dev = ts[0].get_device()
    for t in ts[1:]:
        _require(t.get_device() == dev, f"all tensors must be on {ts[0].device} (got {t.device})")


def _stream_ptr(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


try:  # the current stream's raw handle, without building a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:  # pragma: no cover
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _call(name: str, fn, device: torch.device, *args) -> None:
    """fn(*args, stream) with `device`'s current stream, raising on a non-OK
    status; the device is made current only when it is not already."""
    index = device.index
    if torch.cuda.current_device() == index:
        _capi.check(name, fn(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(index):
            _capi.check(name, fn(*args, _raw_stream(index)))


def _ptr(t: Optional[torch.Tensor]) -> int:
    """Device address of t, or 0 (NULL) for None or an empty tensor."""
    return t.data_ptr() if t is not None and t.numel() > 0 else 0


def _out(out: Optional[torch.Tensor], like_shape, dtype, device, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty(like_shape, dtype=dtype, device=device)
    _cuda(out, name, dtype)
    _require(tuple(out.shape) == tuple(like_shape),
             f"{name} must have shape {tuple(like_shape)} (got {tuple(out.shape)})")
    return out


def _rows_width(x: torch.Tensor, name: str):
    _require(x.dim() >= 2, f"{name} must be [..., width]")
    width = x.shape[-1]
    return x.numel() // width if width else 0, width


# ------------------------------------------------------------------ LN ----

def ln_fwd(x: torch.Tensor, eps: float = 1e-5, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """No-affine LayerNorm over the last dim (192 or 384) of an fp16 or
    bfloat16 tensor."""
    _row16(x, "x")
    rows, width = _rows_width(x, "x")
    _require(width in LN_WIDTHS, f"width must be one of {LN_WIDTHS} (got {width})")
    y = _out(out, x.shape, x.dtype, x.device, "out")
    _same_device(x, y)
    _call("ln_fwd", _entry("ln_fwd", x.dtype), x.device, _ptr(x), _ptr(y), rows, width,
          float(eps))
    return y


def residual_add_ln_fwd(residual: torch.Tensor, branch: torch.Tensor, eps: float = 1e-5,
                        residual_out: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None):
    """Returns (residual_out, y): residual_out = round(residual + branch) in
    the tensors' 16-bit format (fp16 or bfloat16),
    y = LN(residual_out)."""
    _row16(residual, "residual")
    _cuda(branch, "branch", residual.dtype)
    _require(residual.shape == branch.shape, "residual and branch must have the same shape")
    rows, width = _rows_width(residual, "residual")
    _require(width in LN_WIDTHS, f"width must be one of {LN_WIDTHS} (got {width})")
    r = _out(residual_out, residual.shape, residual.dtype, residual.device, "residual_out")
    y = _out(out, residual.shape, residual.dtype, residual.device, "out")
    _same_device(residual, branch, r, y)
    _call("residual_add_ln_fwd", _entry("residual_add_ln_fwd", residual.dtype), residual.device,
          _ptr(residual), _ptr(branch), _ptr(r), _ptr(y), rows, width, float(eps))
    return r, y


# -------------------------------------------------------------- gather ----

def _gather_args(src, idx, out, name):
    _row16(src, "src")
    _cuda(idx, "idx", torch.int32)
    _require(src.dim() == 2, "src must be [n_src, width]")
    _require(idx.dim() == 1, "idx must be 1-D")
    n_src, width = src.shape
    dst = _out(out, (idx.numel(), width), src.dtype, src.device, "out")
    _same_device(src, idx, dst)
    return n_src, width, dst


def window_gather(src: torch.Tensor, idx: torch.Tensor,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dst[d] = src[idx[d]] (idx >= 0) or a zero row (idx == -1).  Rows are
    copied bit for bit, so fp16 and bfloat16 use the same kernel."""
    n_src, width, dst = _gather_args(src, idx, out, "window_gather")
    _call("window_gather", _capi.load().window_gather, src.device,
          _ptr(src), _ptr(idx), _ptr(dst), n_src, idx.numel(), width)
    return dst


def norm_gather(src: torch.Tensor, idx: torch.Tensor, eps: float = 1e-5,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dst[d] = LN(src[idx[d]]) (idx >= 0) or a zero row (idx == -1)."""
    n_src, width, dst = _gather_args(src, idx, out, "norm_gather")
    _require(width in LN_WIDTHS, f"width must be one of {LN_WIDTHS} (got {width})")
    _call("norm_gather", _entry("norm_gather", src.dtype), src.device,
          _ptr(src), _ptr(idx), _ptr(dst), n_src, idx.numel(), width, float(eps))
    return dst


# ------------------------------------------------ block-boundary fusions ----

def window_reverse_add_ln_fwd(residual: torch.Tensor, windows: torch.Tensor,
                              inv_idx: torch.Tensor, eps: float = 1e-5,
                              residual_out: Optional[torch.Tensor] = None,
                              out: Optional[torch.Tensor] = None):
    """Returns (residual_out, y): residual_out[t] = round(residual[t] +
    windows[inv_idx[t]]), y = LN(residual_out)."""
    _row16(residual, "residual")
    _cuda(windows, "windows", residual.dtype)
    _cuda(inv_idx, "inv_idx", torch.int32)
    _require(residual.dim() == 2 and windows.dim() == 2, "residual and windows must be 2-D")
    rows, width = residual.shape
    _require(windows.shape[1] == width, "windows must have the residual's width")
    _require(width in LN_WIDTHS, f"width must be one of {LN_WIDTHS} (got {width})")
    _require(inv_idx.dim() == 1 and inv_idx.numel() == rows, "inv_idx must have one entry per row")
    r = _out(residual_out, residual.shape, residual.dtype, residual.device, "residual_out")
    y = _out(out, residual.shape, residual.dtype, residual.device, "out")
    _same_device(residual, windows, inv_idx, r, y)
    _call("window_reverse_add_ln_fwd", _entry("window_reverse_add_ln_fwd", residual.dtype),
          residual.device, _ptr(residual), _ptr(windows), _ptr(inv_idx), _ptr(r), _ptr(y), rows,
          windows.shape[0], width, float(eps))
    return r, y


def residual_add_norm_gather(residual: torch.Tensor, branch: torch.Tensor, idx: torch.Tensor,
                             eps: float = 1e-5, residual_out: Optional[torch.Tensor] = None,
                             out: Optional[torch.Tensor] = None):
    """Returns (residual_out, dst): residual_out = round(residual + branch),
    dst[d] = LN(residual_out)[idx[d]] (zero row for -1)."""
    _row16(residual, "residual")
    _cuda(branch, "branch", residual.dtype)
    _cuda(idx, "idx", torch.int32)
    _require(residual.shape == branch.shape and residual.dim() == 2,
             "residual and branch must be 2-D and of the same shape")
    n_src, width = residual.shape
    _require(width in LN_WIDTHS, f"width must be one of {LN_WIDTHS} (got {width})")
    _require(idx.dim() == 1, "idx must be 1-D")
    r = _out(residual_out, residual.shape, residual.dtype, residual.device, "residual_out")
    dst = _out(out, (idx.numel(), width), residual.dtype, residual.device, "out")
    _same_device(residual, branch, idx, r, dst)
    _call("residual_add_norm_gather", _entry("residual_add_norm_gather", residual.dtype),
          residual.device, _ptr(residual), _ptr(branch), _ptr(idx), _ptr(r), _ptr(dst), n_src,
          idx.numel(), width, float(eps))
    return r, dst


# ---------------------------------------------------------------- GELU ----

def bias_gelu_tanh(x: torch.Tensor, bias: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gelu_tanh(x + bias) over the last dim, fp32, fp16 or bfloat16."""
    _cuda(x, "x")
    _require(x.dtype in _DTYPE, f"x must be float32, float16 or bfloat16 (got {x.dtype})")
    _cuda(bias, "bias", x.dtype)
    _require(x.dim() >= 1, "x must have at least one dimension")
    width = x.shape[-1]
    _require(bias.dim() == 1 and bias.numel() == width,
             f"bias must be 1-D with {width} elements (got shape {tuple(bias.shape)})")
    rows = x.numel() // width if width else 0
    y = _out(out, x.shape, x.dtype, x.device, "out")
    _same_device(x, bias, y)
    _call("bias_gelu_tanh", _capi.load().bias_gelu_tanh, x.device,
          _ptr(x), _ptr(bias), _ptr(y), rows, width, _DTYPE[x.dtype])
    return y


def gelu_bwd_workspace_bytes(rows: int, width: int) -> int:
    """Bytes of workspace bias_gelu_tanh_bwd needs for a [rows, width] tensor."""
    return int(_capi.load().wgs_bias_gelu_bwd_workspace_bytes(int(rows), int(width)))


def bias_gelu_tanh_bwd(grad_y: torch.Tensor, x: torch.Tensor, bias: torch.Tensor,
                       grad_x: Optional[torch.Tensor] = None,
                       grad_bias: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Backward of gelu_tanh(x + bias).  Returns (grad_x, grad_bias).  The
    deterministic column sum needs a workspace of
    wgs_bias_gelu_bwd_workspace_bytes(rows, width) bytes; one is allocated
    here unless the caller passes a uint8 CUDA tensor that large."""
    _cuda(x, "x")
    _require(x.dtype in _DTYPE, f"x must be float32, float16 or bfloat16 (got {x.dtype})")
    _cuda(grad_y, "grad_y", x.dtype)
    _cuda(bias, "bias", x.dtype)
    _require(grad_y.shape == x.shape and x.dim() >= 1, "grad_y and x must have the same shape")
    width = x.shape[-1]
    _require(bias.dim() == 1 and bias.numel() == width,
             f"bias must be 1-D with {width} elements (got shape {tuple(bias.shape)})")
    rows = x.numel() // width if width else 0
    gx = _out(grad_x, x.shape, x.dtype, x.device, "grad_x")
    gb = _out(grad_bias, bias.shape, x.dtype, x.device, "grad_bias")
    lib = _capi.load()
    need = int(lib.wgs_bias_gelu_bwd_workspace_bytes(rows, width))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _cuda(workspace, "workspace", torch.uint8)
    _same_device(grad_y, x, bias, gx, gb, workspace)
    _call("bias_gelu_tanh_bwd", lib.bias_gelu_tanh_bwd, x.device,
          _ptr(grad_y), _ptr(x), _ptr(bias), _ptr(gx), _ptr(gb), _ptr(workspace),
          workspace.numel(), rows, width, _DTYPE[x.dtype])
    return gx, gb


def window_bias_mask_add(scores: torch.Tensor, bias: torch.Tensor,
                         win_type: Optional[torch.Tensor] = None,
                         region: Optional[torch.Tensor] = None, mask_value: float = -100.0,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention logits plus position bias and shift mask: scores
    [n_win, heads, n, n] (float16 or bfloat16), bias [n_types, heads, n, n],
    win_type int32 [n_win] (None: type 0), region int32 [n_win * n] labels
    (None: no mask).  out may be scores."""
    _row16(scores, "scores")
    _cuda(bias, "bias", scores.dtype)
    _require(scores.dim() == 4 and scores.shape[2] == scores.shape[3],
             f"scores must be [n_win, heads, n, n] (got {tuple(scores.shape)})")
    n_win, heads, n, _ = scores.shape
    _require(bias.dim() == 4 and tuple(bias.shape[1:]) == (heads, n, n),
             f"bias must be [n_types, {heads}, {n}, {n}] (got {tuple(bias.shape)})")
    n_types = bias.shape[0]
    ts = [scores, bias]
    if win_type is not None:
        _cuda(win_type, "win_type", torch.int32)
        _require(win_type.numel() == n_win, f"win_type must have {n_win} entries")
        ts.append(win_type)
    if region is not None:
        _cuda(region, "region", torch.int32)
        _require(region.numel() == n_win * n, f"region must have {n_win * n} entries")
        ts.append(region)
    y = _out(out, scores.shape, scores.dtype, scores.device, "out")
    _same_device(*ts, y)
    _call("window_bias_mask_add", _capi.load().window_bias_mask_add, scores.device,
          _ptr(scores), _ptr(bias), _ptr(win_type), _ptr(region), _ptr(y), n_win, heads, n,
          n_types, float(mask_value), _DTYPE[scores.dtype])
    return y


# The calls below are short next to what Python spends on them, so their
# checks look first and word a message only when something is wrong.

def _fail(msg: str) -> None:
    raise RuntimeError(msg)


_MAX32, _MAX64 = 2 ** 31 - 1, 2 ** 63 - 1


def _int32(v, name: str, most: int = _MAX32) -> int:
    """v as the C ABI takes it: ctypes would cut a larger one silently."""
    v = int(v)
    if not -most - 1 <= v <= most:
        _fail(f"{name} must be at most {most} (got {v})")
    return v


def _int64(v, name: str) -> int:
    return _int32(v, name, _MAX64)


def _given(t: torch.Tensor, name: str, dtype, index: int) -> int:
    """Device address of t (0 when empty), a contiguous tensor of `dtype` on
    CUDA device `index`; raises otherwise."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index
            or not t.is_contiguous()):
        _cuda(t, name, dtype)
        _fail(f"all tensors must be on cuda:{index} (got {name} on {t.device})")
    return t.data_ptr()


def _into(out: Optional[torch.Tensor], shape, dtype, device, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.shape != shape:
        _fail(f"{name} must have shape {tuple(shape)} (got {tuple(out.shape)})")
    return out


def _output(out: Optional[torch.Tensor], shape, dtype, device, name: str, index: int):
    """(the tensor that takes an output, its address): `out` after its checks, or
    a new one, which needs none."""
    if out is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return _into(out, shape, dtype, device, name), _given(out, name, dtype, index)


def _space(workspace: Optional[torch.Tensor], need, device) -> torch.Tensor:
    return workspace if workspace is not None else torch.empty(max(need(), 16), dtype=torch.uint8,
                                                               device=device)


def _run(name: str, fn, index: int, *args) -> None:
    """fn(*args, stream) on device `index`'s current stream."""
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    else:
        status = fn(*args, _raw_stream(index))
    if status:
        _capi.check(name, status)


# ------------------------------------------------------- position bias ----

def window_bucket_count(window: Sequence[int], absolute_axes: int = 0) -> int:
    """Buckets of build_window_buckets: the rows of the learned table."""
    n = _capi.load().wgs_window_bucket_count(_i3(window, "window"),
                                             _int32(absolute_axes, "absolute_axes"))
    _require(n >= 0, "invalid window extents or absolute_axes")
    return int(n)


def build_window_buckets(window: Sequence[int], absolute_axes: int = 0,
                         device=None) -> torch.Tensor:
    """int32 [n, n] bucket map of a window's n cells (host-built); on `device`
    if given.  Axes whose bit is set in absolute_axes keep both positions, the
    others their difference."""
    window_bucket_count(window, absolute_axes)
    n = int(window[0]) * int(window[1]) * int(window[2])
    out = torch.empty(n, n, dtype=torch.int32)
    _capi.check("wgs_build_window_buckets", _capi.load().wgs_build_window_buckets(
        _i3(window, "window"), int(absolute_axes), ctypes.c_void_p(out.data_ptr()), n * n))
    return out if device is None else out.to(device)


def build_distance_buckets(n_q: int, n_k: int, n_buckets: int, max_distance: int,
                           bidirectional: bool = True, q_start: int = 0,
                           device=None) -> torch.Tensor:
    """int32 [n_q, n_k] bucket map of a sequence: single distances, then
    logarithmic ranges up to max_distance (host-built); on `device` if given.
    Query i stands at position q_start + i; without `bidirectional` keys ahead
    of their query have no bucket (-1)."""
    _require(n_q >= 0 and n_k >= 0, "n_q and n_k must not be negative")
    numbers = (_int64(q_start, "q_start"), _int32(n_buckets, "n_buckets"),
               _int32(max_distance, "max_distance"))
    out = torch.empty(n_q, n_k, dtype=torch.int32)
    _capi.check("wgs_build_distance_buckets", _capi.load().wgs_build_distance_buckets(
        n_q, n_k, *numbers, int(bool(bidirectional)), ctypes.c_void_p(out.data_ptr()), n_q * n_k))
    return out if device is None else out.to(device)


def position_bias(table: torch.Tensor, bucket: torch.Tensor, dtype=None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bias[t, h, i, j] = table[t, bucket[i, j], h] (0 for bucket -1): table
    [n_types, n_buckets, heads] (or [n_buckets, heads]: one type), bucket
    int32 [n_q, n_k].  `dtype` is the bias's format, by default out's or the
    table's; the table is float32 or of that format."""
    if not isinstance(table, torch.Tensor) or not table.is_cuda or not table.is_contiguous():
        _cuda(table, "table")
    index = table.get_device()
    where = _given(bucket, "bucket", torch.int32, index)
    dims = table.shape
    if len(dims) not in (2, 3):
        _fail("table must be [n_types, n_buckets, heads] or [n_buckets, heads]")
    if bucket.dim() != 2:
        _fail("bucket must be [n_q, n_k]")
    n_types = dims[0] if len(dims) == 3 else 1
    n_buckets, heads = dims[-2:]
    if max(n_types, n_buckets, heads) > _MAX32:
        _fail(f"n_types, n_buckets and heads must be at most {_MAX32} (got {tuple(dims)})")
    if dtype is None:
        dtype = table.dtype if out is None else out.dtype
    if dtype not in _DTYPE:
        _fail(f"dtype must be float32, float16 or bfloat16 (got {dtype})")
    if table.dtype not in (torch.float32, dtype):
        _fail(f"table must be float32 or {dtype} (got {table.dtype})")
    n_q, n_k = bucket.shape
    y = _into(out, (n_types, heads, n_q, n_k), dtype, table.device, "out")
    _run("position_bias", _capi.load().position_bias, index, table.data_ptr(), where,
         _given(y, "out", dtype, index), n_types, heads, n_q * n_k, n_buckets,
         _DTYPE[table.dtype], _DTYPE[dtype])
    return y


@dataclass(frozen=True)
class BucketPlan:
    """A bucket map's inverse on a device (build_bucket_plan)."""
    words: torch.Tensor      # int32, the C ABI's plan
    shape: tuple             # (n_q, n_k) of the map
    n_buckets: int
    n_slots: int

    @property
    def n_pairs(self) -> int:
        return self.shape[0] * self.shape[1]


def build_bucket_plan(bucket: torch.Tensor, n_buckets: int, device="cuda") -> BucketPlan:
    """The plan that position_bias_bwd reads, from a bucket map int32
    [n_q, n_k] with values in [-1, n_buckets).  Built on one host thread, once
    per map: a map on the GPU is copied back first, which waits for it; about
    13 ms for 1024 x 1024 pairs.  Not for calls under stream capture."""
    _require(isinstance(bucket, torch.Tensor) and bucket.dtype == torch.int32 and bucket.dim() == 2,
             "bucket must be an int32 tensor [n_q, n_k]")
    n_buckets = _int32(n_buckets, "n_buckets")
    host = bucket.cpu().contiguous()
    lib = _capi.load()
    slots = ctypes.c_int64()
    n = lib.wgs_bucket_plan_words(ctypes.c_void_p(host.data_ptr()), host.numel(), n_buckets,
                                  ctypes.byref(slots))
    _require(n >= 0, f"bucket values must lie in [-1, {n_buckets}) and n_buckets be positive")
    words = torch.empty(n, dtype=torch.int32)
    _capi.check("wgs_build_bucket_plan", lib.wgs_build_bucket_plan(
        ctypes.c_void_p(host.data_ptr()), host.numel(), n_buckets,
        ctypes.c_void_p(words.data_ptr()), n))
    return BucketPlan(words.to(device), tuple(host.shape), n_buckets, int(slots.value))


def position_bias_bwd_workspace_bytes(plan: BucketPlan, n_win: int, heads: int,
                                      n_types: int = 1) -> int:
    """Bytes of workspace position_bias_bwd needs."""
    return int(_capi.load().wgs_position_bias_bwd_workspace_bytes(
        _int64(n_win, "n_win"), _int32(heads, "heads"), _int32(n_types, "n_types"), plan.n_pairs,
        plan.n_slots))


def position_bias_bwd(grad: torch.Tensor, plan: BucketPlan,
                      win_type: Optional[torch.Tensor] = None, n_types: int = 1,
                      dtype=torch.float32, grad_table: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of position_bias's table, [n_types, n_buckets, heads], from
    the gradient of the logits grad [n_win, heads, n_q, n_k]; win_type int32
    [n_win] (None: type 0).  `dtype`, the gradient's format, is float32 or
    grad's.  With one type, grad_table may be [n_buckets, heads], as the table
    may, and is returned so.  The fixed-order sums need a workspace of
    position_bias_bwd_workspace_bytes(...) bytes; one is allocated here unless
    the caller passes a uint8 CUDA tensor that large."""
    if not isinstance(grad, torch.Tensor) or not grad.is_cuda or not grad.is_contiguous():
        _cuda(grad, "grad")
    index, kind = grad.get_device(), grad.dtype
    if kind not in _DTYPE:
        _fail(f"grad must be float32, float16 or bfloat16 (got {kind})")
    if not isinstance(plan, BucketPlan):
        _fail("plan must come from build_bucket_plan")
    if grad.dim() != 4 or grad.shape[2:] != plan.shape:
        _fail(f"grad must be [n_win, heads, {plan.shape[0]}, {plan.shape[1]}] (got {tuple(grad.shape)})")
    n_win, heads = grad.shape[:2]
    if n_types < 0:
        _fail("n_types must not be negative")
    if max(n_types, heads) > _MAX32:
        _fail(f"n_types and heads must be at most {_MAX32} (got {n_types}, {heads})")
    if dtype not in (torch.float32, kind):
        _fail(f"dtype must be float32 or {kind} (got {dtype})")
    types = 0
    if win_type is not None:
        types = _given(win_type, "win_type", torch.int32, index)
        if win_type.numel() != n_win:
            _fail(f"win_type must have {n_win} entries")
        if n_win == 0:
            types = 0
    shape = (n_types, plan.n_buckets, heads)
    if grad_table is not None and n_types == 1 and grad_table.dim() == 2:
        shape = shape[1:]
    gt = _into(grad_table, shape, dtype, grad.device, "grad_table")
    ws = _space(workspace, lambda: position_bias_bwd_workspace_bytes(plan, n_win, heads, n_types),
                grad.device)
    _run("position_bias_bwd", _capi.load().position_bias_bwd, index, grad.data_ptr(),
         _given(plan.words, "plan", torch.int32, index), types,
         _given(gt, "grad_table", dtype, index), _given(ws, "workspace", torch.uint8, index),
         ws.numel(), n_win, heads, plan.n_pairs, plan.n_buckets, plan.n_slots, n_types,
         _DTYPE[kind], _DTYPE[dtype])
    return gt


# ---------------------------------------------------------- group norm ----

_ACT = {None: _capi.WGS_ACT_NONE, "none": _capi.WGS_ACT_NONE, "silu": _capi.WGS_ACT_SILU,
        "gelu_tanh": _capi.WGS_ACT_GELU_TANH}


def _norm_args(x, groups, weight, bias, act):
    """(device index, n, spatial, channels, weight's and bias's addresses,
    their dtype) of checked group-norm arguments."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or not x.is_contiguous():
        _cuda(x, "x")
    if x.dtype not in _DTYPE:
        _fail(f"x must be float32, float16 or bfloat16 (got {x.dtype})")
    if act not in _ACT:
        _fail(f"act must be one of {sorted(k for k in _ACT if k)} or None (got {act!r})")
    dims = x.shape
    if len(dims) < 2:
        _fail("x must be [n, ..., channels]")
    n, channels = dims[0], dims[-1]
    if channels <= 0 or groups <= 0 or channels % groups != 0:
        _fail(f"channels ({channels}) must be a multiple of groups ({groups})")
    if channels > _MAX32:
        _fail(f"channels must be at most {_MAX32} (got {channels})")
    spatial = dims[1] if len(dims) == 3 else 1 if len(dims) == 2 else math.prod(dims[1:-1])
    index = x.get_device()
    if weight is None or bias is None:
        if weight is not bias:
            _fail("weight and bias go together")
        return index, n, spatial, channels, 0, 0, torch.float32
    pt = weight.dtype
    if pt is not torch.float32 and pt is not x.dtype:
        _fail(f"weight must be float32 or {x.dtype} (got {pt})")
    w, b = _given(weight, "weight", pt, index), _given(bias, "bias", pt, index)
    if weight.shape != (channels,) or bias.shape != (channels,):
        _fail(f"weight and bias must have {channels} elements")
    return index, n, spatial, channels, w, b, pt


def _norm_sizes(n, spatial, channels, groups):
    return (_int64(n, "n"), _int64(spatial, "spatial"), _int32(channels, "channels"),
            _int32(groups, "groups"))


def group_norm_act_workspace_bytes(n: int, spatial: int, channels: int, groups: int) -> int:
    """Bytes of workspace group_norm_act needs for [n, spatial, channels]."""
    return int(_capi.load().wgs_group_norm_act_workspace_bytes(*_norm_sizes(n, spatial, channels, groups)))


def group_norm_act_bwd_workspace_bytes(n: int, spatial: int, channels: int, groups: int) -> int:
    """Bytes of workspace group_norm_act_bwd needs for [n, spatial, channels]."""
    return int(_capi.load().wgs_group_norm_act_bwd_workspace_bytes(*_norm_sizes(n, spatial, channels, groups)))


def group_norm_act(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   act: Optional[str] = "silu", out: Optional[torch.Tensor] = None,
                   mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Group norm over channels-last x [n, ..., channels] with weight and bias
    [channels] and an activation (None, "silu" or "gelu_tanh").  Returns
    (y, mean, rstd); mean and rstd, float32 [n, groups], are what
    group_norm_act_bwd takes (they are left as they are when x is empty).
    A workspace of group_norm_act_workspace_bytes(...) bytes is allocated here
    unless the caller passes a uint8 CUDA tensor that large."""
    index, n, spatial, channels, w, b, pt = _norm_args(x, groups, weight, bias, act)
    kind, device = x.dtype, x.device
    y = torch.empty_like(x) if out is None else _into(out, x.shape, kind, device, "out")
    m = _into(mean, (n, groups), torch.float32, device, "mean")
    r = _into(rstd, (n, groups), torch.float32, device, "rstd")
    ws = _space(workspace, lambda: group_norm_act_workspace_bytes(n, spatial, channels, groups), device)
    _run("group_norm_act", _capi.load().group_norm_act, index, x.data_ptr(), w, b,
         _given(y, "out", kind, index), _given(m, "mean", torch.float32, index),
         _given(r, "rstd", torch.float32, index), _given(ws, "workspace", torch.uint8, index),
         ws.numel(), n, spatial, channels, groups, float(eps), _ACT[act], _DTYPE[kind], _DTYPE[pt])
    return y, m, r


def group_norm_act_bwd(grad_y: torch.Tensor, x: torch.Tensor, groups: int, mean: torch.Tensor,
                       rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, act: Optional[str] = "silu",
                       grad_x: Optional[torch.Tensor] = None,
                       grad_weight: Optional[torch.Tensor] = None,
                       grad_bias: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Gradients of group_norm_act.  Returns (grad_x, grad_weight, grad_bias),
    the last two None without weight and bias.  grad_x may be grad_y or x."""
    index, n, spatial, channels, w, b, pt = _norm_args(x, groups, weight, bias, act)
    kind, device = x.dtype, x.device
    gy = _given(grad_y, "grad_y", kind, index)
    if grad_y.shape != x.shape:
        _fail("grad_y and x must have the same shape")
    m, r = _given(mean, "mean", torch.float32, index), _given(rstd, "rstd", torch.float32, index)
    if mean.shape != (n, groups) or rstd.shape != (n, groups):
        _fail(f"mean and rstd must have shape {(n, groups)}")
    gx = torch.empty_like(x) if grad_x is None else _into(grad_x, x.shape, kind, device, "grad_x")
    gw = gb = None
    pw = pb = 0
    if weight is not None:
        gw = _into(grad_weight, (channels,), pt, device, "grad_weight")
        gb = _into(grad_bias, (channels,), pt, device, "grad_bias")
        pw, pb = _given(gw, "grad_weight", pt, index), _given(gb, "grad_bias", pt, index)
    elif grad_weight is not None or grad_bias is not None:
        _fail("grad_weight and grad_bias need weight and bias")
    ws = _space(workspace, lambda: group_norm_act_bwd_workspace_bytes(n, spatial, channels, groups),
                device)
    _run("group_norm_act_bwd", _capi.load().group_norm_act_bwd, index, gy, x.data_ptr(), w, b, m, r,
         _given(gx, "grad_x", kind, index), pw, pb, _given(ws, "workspace", torch.uint8, index),
         ws.numel(), n, spatial, channels, groups, _ACT[act], _DTYPE[kind], _DTYPE[pt])
    return gx, gw, gb


# ---------------------------------------------------------- layer norm ----

def _layer_norm_args(x, weight, bias, name):
    """(device index, rows, width, weight's and bias's addresses, their dtype)
    of checked layer-norm arguments."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or not x.is_contiguous():
        _cuda(x, name)
    kind, dims = x.dtype, x.shape
    if kind not in _DTYPE:
        _fail(f"{name} must be float32, float16 or bfloat16 (got {kind})")
    if not dims:
        _fail(f"{name} must be [..., width]")
    width = dims[-1]
    if width > _MAX32:
        _fail(f"the width must be at most {_MAX32} (got {width})")
    rows = dims[0] if len(dims) == 2 else math.prod(dims[:-1])
    index = x.get_device()
    if weight is None:
        if bias is not None:
            _fail("a bias needs a weight")
        return index, rows, width, 0, 0, torch.float32
    pt = weight.dtype if isinstance(weight, torch.Tensor) else None
    if pt is not torch.float32 and pt is not kind:
        _fail(f"weight must be float32 or {kind} (got {pt})")
    w = _given(weight, "weight", pt, index)
    b = _given(bias, "bias", pt, index) if bias is not None else 0
    if weight.shape != (width,) or (b and bias.shape != (width,)):
        _fail(f"weight and bias must have {width} elements")
    return index, rows, width, w, b, pt


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               out: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
               rstd: Optional[torch.Tensor] = None):
    """Layer norm over the last dim (1 to 8192) of a float32, float16 or
    bfloat16 tensor, with weight and bias [width] (float32 or x's format; None:
    1 and 0).  Returns (y, mean, rstd); mean and rstd, float32 and shaped as x
    without its last dim, are what layer_norm_bwd takes."""
    index, rows, width, w, b, pt = _layer_norm_args(x, weight, bias, "x")
    kind, device, shape = x.dtype, x.device, x.shape
    lead = shape[:-1]
    y, py = _output(out, shape, kind, device, "out", index)
    m, pm = _output(mean, lead, torch.float32, device, "mean", index)
    r, pr = _output(rstd, lead, torch.float32, device, "rstd", index)
    _run("layer_norm", _capi.load().layer_norm, index, x.data_ptr(), w, b, py, pm, pr, rows, width,
         float(eps), _DTYPE[kind], _DTYPE[pt])
    return y, m, r


def residual_add_layer_norm(residual: torch.Tensor, branch: torch.Tensor,
                            weight: Optional[torch.Tensor] = None,
                            bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                            residual_out: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None,
                            mean: Optional[torch.Tensor] = None,
                            rstd: Optional[torch.Tensor] = None):
    """Returns (residual_out, y, mean, rstd): residual_out = round(residual +
    branch) in the tensors' format, the others layer_norm's of residual_out."""
    index, rows, width, w, b, pt = _layer_norm_args(residual, weight, bias, "residual")
    kind, device, shape = residual.dtype, residual.device, residual.shape
    second = _given(branch, "branch", kind, index)
    if branch.shape != shape:
        _fail("residual and branch must have the same shape")
    lead = shape[:-1]
    t, to = _output(residual_out, shape, kind, device, "residual_out", index)
    y, py = _output(out, shape, kind, device, "out", index)
    m, pm = _output(mean, lead, torch.float32, device, "mean", index)
    r, pr = _output(rstd, lead, torch.float32, device, "rstd", index)
    _run("residual_add_layer_norm", _capi.load().residual_add_layer_norm, index, residual.data_ptr(),
         second, w, b, to, py, pm, pr, rows, width, float(eps), _DTYPE[kind], _DTYPE[pt])
    return t, y, m, r


def layer_norm_bwd_workspace_bytes(rows: int, width: int) -> int:
    """Bytes of workspace layer_norm_bwd needs for [rows, width]."""
    return int(_capi.load().wgs_layer_norm_bwd_workspace_bytes(_int64(rows, "rows"),
                                                               _int32(width, "width")))


def layer_norm_bwd(grad_y: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: Optional[torch.Tensor] = None,
                   grad_residual: Optional[torch.Tensor] = None,
                   grad_x: Optional[torch.Tensor] = None,
                   grad_weight: Optional[torch.Tensor] = None,
                   grad_bias: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of layer_norm, or of residual_add_layer_norm with x its
    residual_out and grad_residual the gradient that reaches residual_out past
    the norm: grad_x is then that of residual and of branch.  Returns (grad_x,
    grad_weight, grad_bias), the last two in the weight's format, None without
    one.  grad_x may be grad_y, x or grad_residual.  The fixed-order sums need a
    workspace of layer_norm_bwd_workspace_bytes(rows, width) bytes; one is
    allocated here unless the caller passes a uint8 CUDA tensor that large."""
    index, rows, width, w, _, pt = _layer_norm_args(x, weight, None, "x")
    kind, device, shape = x.dtype, x.device, x.shape
    gy = _given(grad_y, "grad_y", kind, index)
    if grad_y.shape != shape:
        _fail("grad_y and x must have the same shape")
    m, r = _given(mean, "mean", torch.float32, index), _given(rstd, "rstd", torch.float32, index)
    if mean.shape != shape[:-1] or rstd.shape != shape[:-1]:
        _fail(f"mean and rstd must have shape {tuple(shape[:-1])}")
    past = 0
    if grad_residual is not None:
        past = _given(grad_residual, "grad_residual", kind, index)
        if grad_residual.shape != shape:
            _fail("grad_residual and x must have the same shape")
    gx, px = _output(grad_x, shape, kind, device, "grad_x", index)
    gw = gb = None
    pw = pb = ws = size = 0
    if weight is not None:
        gw, pw = _output(grad_weight, (width,), pt, device, "grad_weight", index)
        gb, pb = _output(grad_bias, (width,), pt, device, "grad_bias", index)
        space = _space(workspace, lambda: layer_norm_bwd_workspace_bytes(rows, width), device)
        ws, size = _given(space, "workspace", torch.uint8, index), space.numel()
    elif grad_weight is not None or grad_bias is not None:
        _fail("grad_weight and grad_bias need a weight")
    _run("layer_norm_bwd", _capi.load().layer_norm_bwd, index, gy, x.data_ptr(), m, r, w, past, px, pw, pb,
         ws, size, rows, width, _DTYPE[kind], _DTYPE[pt])
    return gx, gw, gb


# ----------------------------------------------------------- embedding ----

def embedding(table: torch.Tensor, idx: torch.Tensor, scale: float = 1.0, dtype=None,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[i] = round(scale * table[idx[i]]) for every entry of idx, int32 of any
    shape (-1: a zero row); table [n_rows, width].  `dtype` is out's format, by
    default out's or the table's; the table is float32 or of that format."""
    if not isinstance(table, torch.Tensor) or not table.is_cuda or not table.is_contiguous():
        _cuda(table, "table")
    index = table.get_device()
    where = _given(idx, "idx", torch.int32, index)
    if table.dim() != 2:
        _fail(f"table must be [n_rows, width] (got {tuple(table.shape)})")
    n_rows, width = table.shape
    if width > _MAX32:
        _fail(f"the width must be at most {_MAX32} (got {width})")
    if dtype is None:
        dtype = table.dtype if out is None else out.dtype
    if dtype not in _DTYPE:
        _fail(f"dtype must be float32, float16 or bfloat16 (got {dtype})")
    if table.dtype not in (torch.float32, dtype):
        _fail(f"table must be float32 or {dtype} (got {table.dtype})")
    y, py = _output(out, (*idx.shape, width), dtype, table.device, "out", index)
    _run("embedding", _capi.load().embedding, index, table.data_ptr(), where, py, idx.numel(), n_rows,
         width, float(scale), _DTYPE[table.dtype], _DTYPE[dtype])
    return y


def embedding_bwd_workspace_bytes(n_idx: int, n_rows: int, width: int) -> int:
    """Bytes of workspace embedding_bwd needs."""
    return int(_capi.load().wgs_embedding_bwd_workspace_bytes(
        _int64(n_idx, "n_idx"), _int64(n_rows, "n_rows"), _int32(width, "width")))


def embedding_bwd(grad: torch.Tensor, idx: torch.Tensor, n_rows: int, scale: float = 1.0,
                  dtype=None, grad_table: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of embedding's table, [n_rows, width], from that of its
    output, grad [*idx.shape, width]: scale times the sum of the rows that idx
    gives to each.  With scale 1 it is window_gather's too.  `dtype`, the
    gradient's format, is float32 or grad's; by default grad_table's, or
    float32.  Sorting idx and the fixed-order sums need a workspace of
    embedding_bwd_workspace_bytes(...) bytes; one is allocated here unless the
    caller passes a uint8 CUDA tensor that large."""
    if not isinstance(grad, torch.Tensor) or not grad.is_cuda or not grad.is_contiguous():
        _cuda(grad, "grad")
    index, kind = grad.get_device(), grad.dtype
    if kind not in _DTYPE:
        _fail(f"grad must be float32, float16 or bfloat16 (got {kind})")
    where = _given(idx, "idx", torch.int32, index)
    width = grad.shape[-1] if grad.dim() else 0
    if grad.dim() != idx.dim() + 1 or grad.shape[:-1] != idx.shape:
        _fail(f"grad must be {(*idx.shape, 'width')} (got {tuple(grad.shape)})")
    if width > _MAX32:
        _fail(f"the width must be at most {_MAX32} (got {width})")
    n_rows = _int64(n_rows, "n_rows")
    if n_rows < 0:
        _fail("n_rows must not be negative")
    if dtype is None:
        dtype = torch.float32 if grad_table is None else grad_table.dtype
    if dtype not in (torch.float32, kind):
        _fail(f"dtype must be float32 or {kind} (got {dtype})")
    n = idx.numel()
    gt, pt = _output(grad_table, (n_rows, width), dtype, grad.device, "grad_table", index)
    ws = _space(workspace, lambda: embedding_bwd_workspace_bytes(n, n_rows, width), grad.device)
    _run("embedding_bwd", _capi.load().embedding_bwd, index, grad.data_ptr(), where,
         pt, _given(ws, "workspace", torch.uint8, index), ws.numel(), n, n_rows, width, float(scale), _DTYPE[kind], _DTYPE[dtype])
    return gt


# ----------------------------------------------------------- index map ----

SHIFT_THEN_PAD, PAD_THEN_SHIFT = 0, 1


def _i3(v, name):
    vals = [_int32(a, name) for a in v]
    _require(len(vals) == 3, f"{name} must have 3 entries")
    return (ctypes.c_int32 * 3)(*vals)


def window_index_count(grid: Sequence[int], window: Sequence[int],
                       padded: Optional[Sequence[int]] = None) -> int:
    n = _capi.load().wgs_window_index_count(_i3(grid, "grid"), _i3(window, "window"),
                                            _i3(padded, "padded") if padded is not None else None)
    _require(n >= 0, "invalid grid / window / padded extents")
    return int(n)


def build_window_index(grid: Sequence[int], window: Sequence[int], shift: Sequence[int],
                       padded: Optional[Sequence[int]] = None, flags: int = SHIFT_THEN_PAD,
                       device=None) -> torch.Tensor:
    """The INT32 destination -> source map (host-built); on `device` if given."""
    n = window_index_count(grid, window, padded)
    out = torch.empty(n, dtype=torch.int32)
    _capi.check("wgs_build_window_index", _capi.load().wgs_build_window_index(
        _i3(grid, "grid"), _i3(window, "window"), _i3(shift, "shift"),
        _i3(padded, "padded") if padded is not None else None, int(flags),
        ctypes.c_void_p(out.data_ptr()), n))
    return out if device is None else out.to(device)


def build_window_inverse(grid: Sequence[int], window: Sequence[int], shift: Sequence[int],
                         padded: Optional[Sequence[int]] = None, flags: int = SHIFT_THEN_PAD,
                         device=None) -> torch.Tensor:
    """inv[t] = the windowed row that holds token t (host-built); on `device` if given."""
    n = 1
    for g in grid:
        n *= int(g)
    out = torch.empty(n, dtype=torch.int32)
    _capi.check("wgs_build_window_inverse", _capi.load().wgs_build_window_inverse(
        _i3(grid, "grid"), _i3(window, "window"), _i3(shift, "shift"),
        _i3(padded, "padded") if padded is not None else None, int(flags),
        ctypes.c_void_p(out.data_ptr()), n))
    return out if device is None else out.to(device)


def build_shift_regions(grid: Sequence[int], window: Sequence[int], shift: Sequence[int],
                        padded: Optional[Sequence[int]] = None, flags: int = SHIFT_THEN_PAD,
                        axes_mask: int = 7, device=None) -> torch.Tensor:
    """INT32 shift-mask region label per windowed row (host-built), in the
    index map's order; on `device` if given."""
    n = window_index_count(grid, window, padded)
    out = torch.empty(n, dtype=torch.int32)
    _capi.check("wgs_build_shift_regions", _capi.load().wgs_build_shift_regions(
        _i3(grid, "grid"), _i3(window, "window"), _i3(shift, "shift"),
        _i3(padded, "padded") if padded is not None else None, int(flags), int(axes_mask),
        ctypes.c_void_p(out.data_ptr()), n))
    return out if device is None else out.to(device)


def check_error(device=None) -> None:
    """Raise WgsError (WGS_ERR_INDEX) if any gather on `device` met an index
    outside [-1, n_src), or any bias-mask add a window type outside
    [0, n_types), or any position-bias call a bucket, window type or plan out
    of its range, or any embedding call an index outside [-1, n_rows), since
    the last check; WGS_ERR_LAUNCH if a kernel gave up
    waiting for its own copies, whose outputs are not to be used (a bad index
    seen too is raised by the next check).  Synchronises that device's current
    stream."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _capi.check("wgs_check_error", _capi.load().wgs_check_error(_stream_ptr(dev)))
