"""Python binding of the steps before the routed experts (ctypes; argument marshalling only).

Names follow the C ABI (include/moe_prologue.h):
  rms_norm_fwd(x, weight, out, eps, residual, residual_out, q, scale, rstd)
  rms_norm_bwd(grad_out, h, weight, rstd, grad_x, grad_weight, workspace, grad_residual)
  moe_router_logits_fwd(x, weight, logits, workspace)
  moe_router_logits_bwd(grad_logits, x, weight, grad_x, grad_weight, workspace)
  moe_route_fwd(logits, ids, weights, bias, score, groups, top_groups, group_score, renormalise, scale)
  moe_route_bwd(grad_weights, logits, ids, grad_logits, score, renormalise, scale)
plus allocating helpers (rms_norm, rms_norm_int8, moe_router_logits, moe_route) and torch.autograd.Function
wrappers (RmsNorm, MoeRouterLogits, MoeRoute), which have first derivatives and refuse a second. Every call
writes into tensors of the caller, on the current stream of their device, and raises TypeError /
ValueError for tensors the C ABI cannot take and MoeEpiError for a status other than success. There
is no fallback.

As in routed.py, each call tests all its tensors in one expression, and looks for the one to name
only when that fails.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import DTYPE_CODE, _handle, _on
from .routed import _code, _fail, _matrix, _refuse, _vector

_F32, _I32, _I8, _U8 = torch.float32, torch.int32, torch.int8, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream
_SCORE = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORE = {"max": 0, "top2": 1}
_fns = None


def _lib():
    """The library with the signatures of this module's calls set."""
    global _fns
    if _fns is None:
        L = binding.lib()
        vp, i64, f32, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
        L.rms_norm_fwd.argtypes = [vp, vp, i32, vp, i32, f32, vp, vp, vp, vp, vp, i64, i64, vp]
        L.rms_norm_bwd.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, i64, i64, i64, vp]
        L.rms_norm_bwd_workspace_bytes.argtypes = [i64, i64]
        L.moe_router_logits_fwd.argtypes = [vp, i32, vp, i32, vp, vp, i64, i64, i64, i64, vp]
        L.moe_router_logits_workspace_bytes.argtypes = [i64, i64, i64]
        L.moe_router_logits_bwd.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, i64, i64, i64, i64, vp]
        L.moe_router_logits_bwd_workspace_bytes.argtypes = [i64, i64, i64]
        L.moe_route_fwd.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, i64, i64, i32, i32, i32, f32, vp]
        L.moe_route_bwd.argtypes = [vp, vp, i32, vp, vp, i64, i64, i64, i32, i32, f32, vp]
        for name in ("rms_norm_fwd", "rms_norm_bwd", "moe_router_logits_fwd", "moe_router_logits_bwd",
                     "moe_route_fwd", "moe_route_bwd"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("rms_norm_bwd_workspace_bytes", "moe_router_logits_workspace_bytes",
                     "moe_router_logits_bwd_workspace_bytes"):
            getattr(L, name).restype = i64
        _fns = L
    return _fns


def _like(t, dtype, shape, device: int) -> bool:
    return t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous()


def _optional(t, name: str, dtype, shape, device: int):
    """The address of a tensor that may be left out (None)."""
    if t is None:
        return None
    if not _like(t, dtype, shape, device):
        _refuse(device, (t, name, dtype, shape))
    return t.data_ptr()


def _space(workspace, device: int):
    """Address and size of a workspace, which may be None."""
    if workspace is None:
        return None, 0
    nbytes = _vector(workspace, "workspace")
    if not (workspace.dtype is _U8 and workspace.get_device() == device and workspace.is_contiguous()):
        _refuse(device, (workspace, "workspace", _U8, None))
    return workspace.data_ptr(), nbytes


def _weight_code(weight, name: str, dtype) -> int:
    """The dtype code of a weight, which is of the rows' type or float32."""
    code = _code(weight, name)
    if weight.dtype is not dtype and weight.dtype is not _F32:
        raise TypeError(f"{name}: expected {dtype} or float32, got {weight.dtype}")
    return code


def _choice(table, value, name: str) -> int:
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name}: expected one of {', '.join(table)}, got {value!r}")
    return code


def _bytes(call: str, **sizes) -> int:
    n = getattr(_lib(), call + "_workspace_bytes")(*(int(v) for v in sizes.values()))
    if n < 0:
        raise ValueError(f"{call} takes no {', '.join(f'{k}={v}' for k, v in sizes.items())}")
    return n


# ---- norm ---------------------------------------------------------------------------

def rms_norm_fwd(x, weight, out, eps: float, residual=None, residual_out=None, q=None, scale=None, rstd=None,
                 stream=None) -> None:
    """h = x + residual (rounded to x's dtype), y = h / sqrt(mean(h^2) + eps) * weight. x [rows, cols] (bf16, fp16
    or fp32); weight [cols] of x's dtype or fp32; out like x, or None if q is given; residual like x, or None;
    residual_out like x for h, or None, and may be residual itself; q int8 [rows, cols] with scale fp32 [rows] for
    y in 8-bit integers (of quantize_rows_int8_fwd's form), or both None; rstd fp32 [rows] for the gradient, or
    None."""
    rows, cols = shape = _matrix(x, "x")
    dev, dt, code, w_code = x.get_device(), x.dtype, _code(x, "x"), _weight_code(weight, "weight", x.dtype)
    if not (dev >= 0 and x.is_contiguous() and _like(weight, weight.dtype, (cols,), dev)):
        _refuse(dev, (x, "x", dt, None), (weight, "weight", weight.dtype, (cols,)))
    if out is None and q is None:
        raise ValueError("out is required where q is None")
    if (q is None) != (scale is None):
        raise ValueError("q and scale go together")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out goes with a residual")
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).rms_norm_fwd, x.data_ptr(), _optional(residual, "residual", dt, shape, dev), code,
                 weight.data_ptr(), w_code, eps, _optional(out, "out", dt, shape, dev),
                 _optional(residual_out, "residual_out", dt, shape, dev), _optional(q, "q", _I8, shape, dev),
                 _optional(scale, "scale", _F32, (rows,), dev), _optional(rstd, "rstd", _F32, (rows,), dev), rows, cols,
                 handle)
    if status:
        _fail(status, "rms_norm_fwd")


def rms_norm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    """Bytes of workspace that rms_norm_bwd needs for a grad_weight."""
    return _bytes("rms_norm_bwd", rows=rows, cols=cols)


def rms_norm_bwd(grad_out, h, weight, rstd, grad_x, grad_weight=None, workspace=None, grad_residual=None,
                 stream=None) -> None:
    """grad_x = rstd * (g - a * mean(g * a)) + grad_residual with a = h * rstd, g = grad_out * weight (the gradient of
    x and of the residual); grad_weight = the sum over the rows of grad_out * a, or None. h is rms_norm_fwd's
    residual_out, or x where it had no residual; grad_residual is the gradient of residual_out, or None. grad_weight
    of weight's dtype; workspace uint8 of rms_norm_bwd_workspace_bytes, or None if grad_weight is."""
    rows, cols = shape = _matrix(h, "h")
    dev, dt, code, w_code = h.get_device(), h.dtype, _code(h, "h"), _weight_code(weight, "weight", h.dtype)
    if not (dev >= 0 and h.is_contiguous() and _like(weight, weight.dtype, (cols,), dev)
            and grad_out is not None and _like(grad_out, dt, shape, dev)
            and rstd is not None and _like(rstd, _F32, (rows,), dev)
            and grad_x is not None and _like(grad_x, dt, shape, dev)):
        _refuse(dev, (h, "h", dt, None), (weight, "weight", weight.dtype, (cols,)), (grad_out, "grad_out", dt, shape),
                (rstd, "rstd", _F32, (rows,)), (grad_x, "grad_x", dt, shape))
    ws, nbytes = _space(workspace, dev)
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).rms_norm_bwd, grad_out.data_ptr(), h.data_ptr(), code, weight.data_ptr(), w_code,
                 rstd.data_ptr(), _optional(grad_residual, "grad_residual", dt, shape, dev), grad_x.data_ptr(),
                 _optional(grad_weight, "grad_weight", weight.dtype, (cols,), dev), ws, nbytes, rows, cols, handle)
    if status:
        _fail(status, "rms_norm_bwd")


def _rows(t, name: str, like=None):
    """t as contiguous rows [-1, cols]."""
    if t is None:
        return None
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name}: expected shape {tuple(like.shape)}, got {tuple(t.shape)}")
    if not t.dim():
        raise ValueError(f"{name} must have rows")
    return t.reshape(-1, t.shape[-1]).contiguous()


def rms_norm(x, weight, eps: float, residual=None):
    """y of rms_norm_fwd in a new tensor, and with a residual (y, h). x [..., cols]. No gradients (RmsNorm has
    them)."""
    rows, stream = _rows(x, "x"), _rows(residual, "residual", x)
    out = torch.empty_like(rows)
    h = None if stream is None else torch.empty_like(rows)
    rms_norm_fwd(rows, weight, out, eps, residual=stream, residual_out=h)
    return out.view(x.shape) if h is None else (out.view(x.shape), h.view(x.shape))


def rms_norm_int8(x, weight, eps: float, residual=None):
    """(q, scale) of rms_norm_fwd in new tensors, and with a residual (q, scale, h). x [..., cols]."""
    rows, stream = _rows(x, "x"), _rows(residual, "residual", x)
    q = torch.empty(rows.shape, dtype=_I8, device=x.device)
    scale = torch.empty(rows.shape[0], dtype=_F32, device=x.device)
    h = None if stream is None else torch.empty_like(rows)
    rms_norm_fwd(rows, weight, None, eps, residual=stream, residual_out=h, q=q, scale=scale)
    found = (q.view(x.shape), scale.view(x.shape[:-1]))
    return found if h is None else (*found, h.view(x.shape))


class RmsNorm(torch.autograd.Function):
    """The norm of rows [rows, cols]: RmsNorm.apply(x, weight, eps) is y, RmsNorm.apply(x, weight, eps, residual) is
    (y, h). First derivatives only."""

    @staticmethod
    def forward(ctx, x, weight, eps, residual=None):
        ctx.set_materialize_grads(False)
        x, weight = x.contiguous(), weight.contiguous()
        residual = None if residual is None else residual.contiguous()
        out, rstd = torch.empty_like(x), torch.empty(x.shape[0], dtype=_F32, device=x.device)
        h = None if residual is None else torch.empty_like(x)
        rms_norm_fwd(x, weight, out, eps, residual=residual, residual_out=h, rstd=rstd)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        return out if h is None else (out, h)

    @staticmethod
    def backward(ctx, grad_out, grad_h=None):
        if grad_out is None:                       # the normed rows are not used: the sum's gradient is passed on
            return grad_h, None, None, grad_h
        binding._first_derivative_only("RmsNorm", True)   # the gradients depend on the rows and on the weight
        h, weight, rstd = ctx.saved_tensors
        grad_x = torch.empty_like(h)
        grad_weight = workspace = None
        if ctx.needs_input_grad[1]:
            grad_weight = torch.empty_like(weight)
            workspace = torch.empty(rms_norm_bwd_workspace_bytes(*h.shape), dtype=_U8, device=h.device)
        rms_norm_bwd(grad_out.contiguous(), h, weight, rstd, grad_x, grad_weight, workspace,
                     grad_residual=None if grad_h is None else grad_h.contiguous())
        return grad_x, grad_weight, None, grad_x if any(ctx.needs_input_grad[3:]) else None


# ---- the router's product -----------------------------------------------------------------

def moe_router_logits_workspace_bytes(tokens: int, hidden: int, experts: int) -> int:
    """Bytes of workspace that moe_router_logits_fwd needs for these sizes (0: it may be None)."""
    return _bytes("moe_router_logits", tokens=tokens, hidden=hidden, experts=experts)


def moe_router_logits_fwd(x, weight, logits, workspace=None, stream=None) -> None:
    """logits[t, e] = the fp32 sum of x[t] * weight[e]. x [tokens, hidden] (bf16, fp16 or fp32); weight [experts,
    hidden] of x's dtype or fp32; logits fp32 [tokens, experts]; workspace uint8 of
    moe_router_logits_workspace_bytes, or None if that is 0."""
    tokens, hidden = _matrix(x, "x")
    experts = _matrix(weight, "weight")[0]
    dev, dt, code, w_code = x.get_device(), x.dtype, _code(x, "x"), _weight_code(weight, "weight", x.dtype)
    if not (dev >= 0 and x.is_contiguous() and _like(weight, weight.dtype, (experts, hidden), dev)
            and logits is not None and _like(logits, _F32, (tokens, experts), dev)):
        _refuse(dev, (x, "x", dt, None), (weight, "weight", weight.dtype, (experts, hidden)),
                (logits, "logits", _F32, (tokens, experts)))
    ws, nbytes = _space(workspace, dev)
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_router_logits_fwd, x.data_ptr(), code, weight.data_ptr(), w_code,
                 logits.data_ptr(), ws, nbytes, tokens, hidden, experts, handle)
    if status:
        _fail(status, "moe_router_logits_fwd")


def moe_router_logits_bwd_workspace_bytes(tokens: int, hidden: int, experts: int) -> int:
    """Bytes of workspace that moe_router_logits_bwd needs for a grad_weight (0: it may be None)."""
    return _bytes("moe_router_logits_bwd", tokens=tokens, hidden=hidden, experts=experts)


def moe_router_logits_bwd(grad_logits, x, weight, grad_x, grad_weight, workspace=None, stream=None) -> None:
    """grad_x[t] = the sum of grad_logits[t, e] * weight[e], grad_weight[e] = the sum of grad_logits[t, e] * x[t].
    grad_logits fp32 [tokens, experts]; grad_x like x, grad_weight like weight; either may be None. workspace uint8
    of moe_router_logits_bwd_workspace_bytes, or None if that is 0 or grad_weight is None."""
    tokens, hidden = _matrix(x, "x")
    experts = _matrix(weight, "weight")[0]
    dev, dt, code, w_code = x.get_device(), x.dtype, _code(x, "x"), _weight_code(weight, "weight", x.dtype)
    if not (dev >= 0 and x.is_contiguous() and _like(weight, weight.dtype, (experts, hidden), dev)
            and grad_logits is not None and _like(grad_logits, _F32, (tokens, experts), dev)):
        _refuse(dev, (x, "x", dt, None), (weight, "weight", weight.dtype, (experts, hidden)),
                (grad_logits, "grad_logits", _F32, (tokens, experts)))
    if grad_x is None and grad_weight is None:
        raise ValueError("grad_x or grad_weight is required")
    ws, nbytes = _space(workspace, dev)
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_router_logits_bwd, grad_logits.data_ptr(), x.data_ptr(), code,
                 weight.data_ptr(), w_code, _optional(grad_x, "grad_x", dt, (tokens, hidden), dev),
                 _optional(grad_weight, "grad_weight", weight.dtype, (experts, hidden), dev), ws, nbytes, tokens, hidden,
                 experts, handle)
    if status:
        _fail(status, "moe_router_logits_bwd")


def moe_router_logits(x, weight):
    """The logits of moe_router_logits_fwd in a new tensor."""
    tokens, hidden = _matrix(x, "x")
    experts = _matrix(weight, "weight")[0]
    logits = torch.empty((tokens, experts), dtype=_F32, device=x.device)
    workspace = torch.empty(moe_router_logits_workspace_bytes(tokens, hidden, experts), dtype=_U8, device=x.device)
    moe_router_logits_fwd(x.contiguous(), weight.contiguous(), logits, workspace)
    return logits


class MoeRouterLogits(torch.autograd.Function):
    """The router's product: MoeRouterLogits.apply(x, weight). First derivatives only."""

    @staticmethod
    def forward(ctx, x, weight):
        x, weight = x.contiguous(), weight.contiguous()
        ctx.save_for_backward(x, weight)
        return moe_router_logits(x, weight)

    @staticmethod
    def backward(ctx, grad_logits):
        # each gradient is linear in grad_logits and in the other input
        again = grad_logits.requires_grad or (ctx.needs_input_grad[0] and ctx.needs_input_grad[1])
        binding._first_derivative_only("MoeRouterLogits", again)
        x, weight = ctx.saved_tensors
        grad_x = torch.empty_like(x) if ctx.needs_input_grad[0] else None
        grad_weight = workspace = None
        if ctx.needs_input_grad[1]:
            grad_weight = torch.empty_like(weight)
            workspace = torch.empty(moe_router_logits_bwd_workspace_bytes(*x.shape, weight.shape[0]), dtype=_U8,
                                    device=x.device)
        moe_router_logits_bwd(grad_logits.contiguous(), x, weight, grad_x, grad_weight, workspace)
        return grad_x, grad_weight


# ---- choice of the experts ---------------------------------------------------------------------

def moe_route_fwd(logits, ids, weights, bias=None, score: str = "softmax", groups: int = 1, top_groups: int = 1,
                  group_score: str = "max", renormalise: bool = True, scale: float = 1.0, stream=None) -> None:
    """The top_k experts of each token by s + bias, s = softmax or sigmoid of the logits, in descending order and the
    lowest first of equal ones, and their weights scale * s, over the sum of the chosen s if renormalise. logits
    [tokens, experts] (bf16, fp16 or fp32); ids int32 and weights fp32 [tokens, top_k]; bias fp32 [experts] or None.
    With groups of experts, only those of the top_groups best are chosen from; a group counts for its best expert
    ("max") or the sum of its two best ("top2"). Experts with a logit or bias of -inf or NaN are not chosen: ids -1
    and weight 0 where fewer remain."""
    tokens, experts = _matrix(logits, "logits")
    top_k = _matrix(ids, "ids")[1]
    dev, code, slots = logits.get_device(), _code(logits, "logits"), (tokens, top_k)
    score_code, group_code = _choice(_SCORE, score, "score"), _choice(_GROUP_SCORE, group_score, "group_score")
    if not (dev >= 0 and logits.is_contiguous() and _like(ids, _I32, slots, dev)
            and weights is not None and _like(weights, _F32, slots, dev)):
        _refuse(dev, (logits, "logits", logits.dtype, None), (ids, "ids", _I32, slots),
                (weights, "weights", _F32, slots))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_route_fwd, logits.data_ptr(), code,
                 _optional(bias, "bias", _F32, (experts,), dev), ids.data_ptr(), weights.data_ptr(), tokens, experts,
                 top_k, groups, top_groups, score_code, group_code, 1 if renormalise else 0, scale, handle)
    if status:
        _fail(status, "moe_route_fwd")


def moe_route_bwd(grad_weights, logits, ids, grad_logits, score: str = "softmax", renormalise: bool = True,
                  scale: float = 1.0, stream=None) -> None:
    """grad_logits of the weights of moe_route_fwd, its ids being fixed. grad_weights fp32 and ids int32 [tokens,
    top_k]; logits and grad_logits [tokens, experts] of one dtype. Slots whose id is no expert have no part."""
    tokens, experts = _matrix(logits, "logits")
    top_k = _matrix(ids, "ids")[1]
    dev, dt, code, slots = logits.get_device(), logits.dtype, _code(logits, "logits"), (tokens, top_k)
    score_code = _choice(_SCORE, score, "score")
    if not (dev >= 0 and logits.is_contiguous() and _like(ids, _I32, slots, dev)
            and grad_weights is not None and _like(grad_weights, _F32, slots, dev)
            and grad_logits is not None and _like(grad_logits, dt, (tokens, experts), dev)):
        _refuse(dev, (logits, "logits", dt, None), (ids, "ids", _I32, slots),
                (grad_weights, "grad_weights", _F32, slots), (grad_logits, "grad_logits", dt, (tokens, experts)))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_route_bwd, grad_weights.data_ptr(), logits.data_ptr(), code, ids.data_ptr(),
                 grad_logits.data_ptr(), tokens, experts, top_k, score_code, 1 if renormalise else 0, scale, handle)
    if status:
        _fail(status, "moe_route_bwd")


def moe_route(logits, top_k: int, bias=None, score: str = "softmax", groups: int = 1, top_groups: int = 1,
              group_score: str = "max", renormalise: bool = True, scale: float = 1.0):
    """(ids, weights) of moe_route_fwd in new tensors. No gradients (MoeRoute has them)."""
    tokens = _matrix(logits, "logits")[0]
    ids = torch.empty((tokens, top_k), dtype=_I32, device=logits.device)
    weights = torch.empty((tokens, top_k), dtype=_F32, device=logits.device)
    moe_route_fwd(logits.contiguous(), ids, weights, bias, score, groups, top_groups, group_score, renormalise, scale)
    return ids, weights


class MoeRoute(torch.autograd.Function):
    """The choice of the experts: MoeRoute.apply(logits, top_k, bias=None, score="softmax", groups=1, top_groups=1,
    group_score="max", renormalise=True, scale=1.0) is (ids, weights). The logits have a gradient, from the weights;
    the bias has none. First derivatives only."""

    @staticmethod
    def forward(ctx, logits, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_score="max",
                renormalise=True, scale=1.0):
        logits = logits.contiguous()
        ids, weights = moe_route(logits, top_k, bias, score, groups, top_groups, group_score, renormalise, scale)
        ctx.save_for_backward(logits, ids)
        ctx.form = score, renormalise, scale
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    def backward(ctx, _, grad_weights):
        # the gradient depends on the logits, whose gradient is being taken
        binding._first_derivative_only("MoeRoute", True)
        logits, ids = ctx.saved_tensors
        grad_logits = torch.empty_like(logits)
        moe_route_bwd(grad_weights.contiguous(), logits, ids, grad_logits, *ctx.form)
        return (grad_logits,) + (None,) * 8
