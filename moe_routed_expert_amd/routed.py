"""Python binding of the steps around the routed experts (ctypes; argument marshalling only).

Names follow the C ABI (include/moe_routed.h):
  moe_sort_fwd(expert_of, first_expert, offs, row_of, slot_of, workspace)
  moe_dispatch_fwd(x, slot_of, top_k, out)
  moe_dispatch_bwd(grad_out, row_of, grad_x)
  moe_combine_weighted_fwd(expert_out, row_of, weights, out)
  moe_combine_weighted_bwd(grad_out, expert_out, row_of, weights, grad_expert_out, grad_weights)
  quantize_rows_int8_fwd(x, q, scale)
  grouped_gate_up_swiglu_int8_fwd(a, a_scale, slot_of, top_k, w_gate, w_gate_scale, w_up, w_up_scale, offs, probs,
                                  y, limit)
  grouped_down_router_int8_fwd(h, h_scale, w_down, w_down_scale, offs, probs, out)
plus allocating helpers (moe_sort, quantize_rows_int8) and torch.autograd.Function wrappers
(MoeDispatch, MoeCombineWeighted), which have first derivatives and refuse a second. Every call
writes into tensors of the caller, on the current stream of their device, and raises TypeError /
ValueError for tensors the C ABI cannot take and MoeEpiError for a status other than success. There
is no fallback.

These calls are also made for single tokens, where a kernel runs for a few microseconds, so each
call tests all its tensors in one expression, and looks for the one to name only when that fails.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import DTYPE_CODE, MoeEpiError, _handle, _on

_BF16, _F32, _I32, _I64, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.int8
_raw_stream = torch._C._cuda_getCurrentRawStream
_fns = None


def _lib():
    """The library with the signatures of this module's calls set."""
    global _fns
    if _fns is None:
        L = binding.lib()
        vp, i64, f32, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
        L.moe_sort_fwd.argtypes = [vp, i32, i64, vp, vp, vp, vp, i64, i64, i64, i64, vp]
        L.moe_sort_workspace_bytes.argtypes = [i64, i64, i64]
        L.moe_dispatch_fwd.argtypes = [vp, i32, vp, vp, i64, i64, i64, i64, vp]
        L.moe_dispatch_bwd.argtypes = [vp, i32, vp, vp, i64, i64, i64, i64, vp]
        L.moe_combine_weighted_fwd.argtypes = [vp, i32, vp, vp, vp, i32, i64, i64, i64, i64, vp]
        L.moe_combine_weighted_bwd.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i64, i64, i64, i64, vp]
        L.quantize_rows_int8_fwd.argtypes = [vp, i32, vp, vp, i64, i64, vp]
        L.grouped_gate_up_swiglu_int8_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                                      i64, f32, vp]
        L.grouped_down_router_int8_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, i64, vp]
        for name in ("moe_sort_fwd", "moe_dispatch_fwd", "moe_dispatch_bwd", "moe_combine_weighted_fwd",
                     "moe_combine_weighted_bwd", "quantize_rows_int8_fwd", "grouped_gate_up_swiglu_int8_fwd",
                     "grouped_down_router_int8_fwd"):
            getattr(L, name).restype = ctypes.c_int
        L.moe_sort_workspace_bytes.restype = i64
        _fns = L
    return _fns


def _refuse(device: int, *tensors) -> None:
    """Say which of (tensor, name, dtype, shape) is not contiguous, of this dtype and shape (None: any) and on this
    GPU. Called when a call's own short test of all its tensors has failed."""
    where = torch.device("cuda", device) if device >= 0 else torch.device("cuda")
    for t, name, dtype, shape in tensors:
        binding._need(t, name, dtype, [() if t is None else t.shape if shape is None else shape], where)
    raise ValueError(f"expected tensors on {where}")


def _missing(name: str) -> None:
    raise ValueError(f"{name} is required")


def _code(t: torch.Tensor, name: str) -> int:
    if t is None:
        _missing(name)
    code = DTYPE_CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    return code


def _matrix(t: torch.Tensor, name: str):
    if t is None:
        _missing(name)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(shape)}")
    return shape


def _vector(t: torch.Tensor, name: str) -> int:
    if t is None:
        _missing(name)
    shape = t.shape
    if len(shape) != 1:
        raise ValueError(f"{name} must be 1-D, got {tuple(shape)}")
    return shape[0]


def _experts(w: torch.Tensor, name: str):
    if w is None:
        _missing(name)
    shape = w.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be 3-D [experts, out, in], got {tuple(shape)}")
    return shape


def _optional(t, name: str, dtype, rows: int, device: int):
    """The address of a vector of `rows` values that may be left out (None)."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.get_device() == device and t.shape == (rows,) and t.is_contiguous()):
        _refuse(device, (t, name, dtype, (rows,)))
    return t.data_ptr()


def _fail(status: int, where: str) -> None:
    raise MoeEpiError(status, where)


# ---- order of the rows ------------------------------------------------------------

def moe_sort_workspace_bytes(tokens: int, top_k: int, experts: int) -> int:
    """Bytes of workspace that moe_sort_fwd needs for these sizes (0: it may be None)."""
    n = _lib().moe_sort_workspace_bytes(int(tokens), int(top_k), int(experts))
    if n < 0:
        raise ValueError(f"moe_sort_fwd takes no tokens={tokens}, top_k={top_k}, experts={experts}")
    return n


def moe_sort_fwd(expert_of, first_expert: int, offs, row_of, slot_of, workspace=None, stream=None) -> None:
    """Order of the routed rows. expert_of [tokens, top_k] int32 or int64; the experts of this GPU are
    [first_expert, first_expert + len(offs)). offs int32 [experts] cumulative row counts; row_of int32
    [tokens, top_k] the row of each slot or -1; slot_of int32 [tokens * top_k] the slot of each row, -1
    past the last; workspace uint8 of moe_sort_workspace_bytes, or None if that is 0."""
    tokens, top_k = _matrix(expert_of, "expert_of")
    dev, dt, experts = expert_of.get_device(), expert_of.dtype, _vector(offs, "offs")
    if not (dev >= 0 and (dt is _I32 or dt is _I64) and expert_of.is_contiguous()
            and offs.dtype is _I32 and offs.get_device() == dev and offs.is_contiguous()
            and row_of is not None and row_of.dtype is _I32 and row_of.get_device() == dev
            and row_of.shape == (tokens, top_k) and row_of.is_contiguous()
            and slot_of is not None and slot_of.dtype is _I32 and slot_of.get_device() == dev
            and slot_of.shape == (tokens * top_k,) and slot_of.is_contiguous()):
        _refuse(dev, (expert_of, "expert_of", _I64 if dt is _I64 else _I32, None), (offs, "offs", _I32, None),
                (row_of, "row_of", _I32, (tokens, top_k)), (slot_of, "slot_of", _I32, (tokens * top_k,)))
    ws, nbytes = None, 0
    if workspace is not None:
        nbytes = _vector(workspace, "workspace")
        if not (workspace.dtype is torch.uint8 and workspace.get_device() == dev and workspace.is_contiguous()):
            _refuse(dev, (workspace, "workspace", torch.uint8, None))
        ws = workspace.data_ptr()
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_sort_fwd, expert_of.data_ptr(), 8 if dt is _I64 else 4, first_expert,
                 offs.data_ptr(), row_of.data_ptr(), slot_of.data_ptr(), ws, nbytes, tokens, top_k, experts, handle)
    if status:
        _fail(status, "moe_sort_fwd")


def moe_sort(expert_of, experts: int, first_expert: int = 0):
    """(offs, row_of, slot_of) of moe_sort_fwd in new tensors."""
    tokens, top_k = _matrix(expert_of, "expert_of")
    dev = expert_of.device
    offs = torch.empty(experts, dtype=_I32, device=dev)
    row_of = torch.empty((tokens, top_k), dtype=_I32, device=dev)
    slot_of = torch.empty(tokens * top_k, dtype=_I32, device=dev)
    workspace = torch.empty(moe_sort_workspace_bytes(tokens, top_k, experts), dtype=torch.uint8, device=dev)
    moe_sort_fwd(expert_of.contiguous(), first_expert, offs, row_of, slot_of, workspace)
    return offs, row_of, slot_of


# ---- moves of the rows ---------------------------------------------------------------

def moe_dispatch_fwd(x, slot_of, top_k: int, out, stream=None) -> None:
    """out[r] = x[slot_of[r] // top_k] for every row r whose slot is in range, zeros for the others. x [tokens,
    hidden], out [rows, hidden] of x's dtype (bf16, fp16 or fp32); slot_of int32 [rows]."""
    tokens, hidden = _matrix(x, "x")
    rows, dev, dt, code = _vector(slot_of, "slot_of"), x.get_device(), x.dtype, _code(x, "x")
    if not (dev >= 0 and x.is_contiguous()
            and slot_of.dtype is _I32 and slot_of.get_device() == dev and slot_of.is_contiguous()
            and out is not None and out.dtype is dt and out.get_device() == dev and out.shape == (rows, hidden)
            and out.is_contiguous()):
        _refuse(dev, (x, "x", dt, None), (slot_of, "slot_of", _I32, None), (out, "out", dt, (rows, hidden)))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_dispatch_fwd, x.data_ptr(), code, slot_of.data_ptr(), out.data_ptr(), rows,
                 tokens, top_k, hidden, handle)
    if status:
        _fail(status, "moe_dispatch_fwd")


def moe_dispatch_bwd(grad_out, row_of, grad_x, stream=None) -> None:
    """grad_x[t] = the fp32 sum of grad_out[row_of[t, j]] over the slots that have a row, rounded once.
    grad_out [rows, hidden], grad_x [tokens, hidden] of one dtype; row_of int32 [tokens, top_k]."""
    rows, hidden = _matrix(grad_out, "grad_out")
    tokens, top_k = _matrix(row_of, "row_of")
    dev, dt, code = grad_out.get_device(), grad_out.dtype, _code(grad_out, "grad_out")
    if not (dev >= 0 and grad_out.is_contiguous()
            and row_of.dtype is _I32 and row_of.get_device() == dev and row_of.is_contiguous()
            and grad_x is not None and grad_x.dtype is dt and grad_x.get_device() == dev
            and grad_x.shape == (tokens, hidden) and grad_x.is_contiguous()):
        _refuse(dev, (grad_out, "grad_out", dt, None), (row_of, "row_of", _I32, None),
                (grad_x, "grad_x", dt, (tokens, hidden)))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_dispatch_bwd, grad_out.data_ptr(), code, row_of.data_ptr(),
                 grad_x.data_ptr(), rows, tokens, top_k, hidden, handle)
    if status:
        _fail(status, "moe_dispatch_bwd")


def moe_combine_weighted_fwd(expert_out, row_of, weights, out, stream=None) -> None:
    """out[t] = the fp32 sum of weights[t, j] * expert_out[row_of[t, j]] over the slots that have a row,
    rounded once. expert_out [rows, hidden] (bf16, fp16 or fp32); row_of int32 and weights fp32
    [tokens, top_k]; out [tokens, hidden] of expert_out's dtype or fp32."""
    rows, hidden = _matrix(expert_out, "expert_out")
    tokens, top_k = _matrix(row_of, "row_of")
    dev, code, out_code = expert_out.get_device(), _code(expert_out, "expert_out"), _code(out, "out")
    if not (dev >= 0 and expert_out.is_contiguous()
            and row_of.dtype is _I32 and row_of.get_device() == dev and row_of.is_contiguous()
            and weights is not None and weights.dtype is _F32 and weights.get_device() == dev
            and weights.shape == (tokens, top_k) and weights.is_contiguous()
            and out.get_device() == dev and out.shape == (tokens, hidden) and out.is_contiguous()):
        _refuse(dev, (expert_out, "expert_out", expert_out.dtype, None), (row_of, "row_of", _I32, None),
                (weights, "weights", _F32, (tokens, top_k)), (out, "out", out.dtype, (tokens, hidden)))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_combine_weighted_fwd, expert_out.data_ptr(), code, row_of.data_ptr(),
                 weights.data_ptr(), out.data_ptr(), out_code, rows, tokens, top_k, hidden, handle)
    if status:
        _fail(status, "moe_combine_weighted_fwd")


def moe_combine_weighted_bwd(grad_out, expert_out, row_of, weights, grad_expert_out, grad_weights,
                             stream=None) -> None:
    """grad_expert_out[row_of[t, j]] = weights[t, j] * grad_out[t]; grad_weights[t, j] = the dot product of
    grad_out[t] and expert_out[row_of[t, j]] (fp32), 0 for a slot without a row. grad_out of expert_out's
    dtype or fp32. expert_out and grad_weights may both be None (weights without gradient)."""
    tokens, hidden = _matrix(grad_out, "grad_out")
    top_k = _matrix(row_of, "row_of")[1]
    rows, dt, dev = _matrix(grad_expert_out, "grad_expert_out")[0], grad_expert_out.dtype, grad_out.get_device()
    code, grad_code, slots = _code(grad_expert_out, "grad_expert_out"), _code(grad_out, "grad_out"), (tokens, top_k)
    if not (dev >= 0 and grad_out.is_contiguous()
            and row_of.dtype is _I32 and row_of.get_device() == dev and row_of.shape == slots
            and row_of.is_contiguous()
            and weights is not None and weights.dtype is _F32 and weights.get_device() == dev
            and weights.shape == slots and weights.is_contiguous()
            and grad_expert_out.get_device() == dev and grad_expert_out.shape == (rows, hidden)
            and grad_expert_out.is_contiguous()):
        _refuse(dev, (grad_out, "grad_out", grad_out.dtype, None), (row_of, "row_of", _I32, slots),
                (weights, "weights", _F32, slots), (grad_expert_out, "grad_expert_out", dt, (rows, hidden)))
    eo = gw = None
    if grad_weights is not None:
        if not (expert_out is not None and expert_out.dtype is dt and expert_out.get_device() == dev
                and expert_out.shape == (rows, hidden) and expert_out.is_contiguous()
                and grad_weights.dtype is _F32 and grad_weights.get_device() == dev
                and grad_weights.shape == slots and grad_weights.is_contiguous()):
            _refuse(dev, (expert_out, "expert_out", dt, (rows, hidden)), (grad_weights, "grad_weights", _F32, slots))
        eo, gw = expert_out.data_ptr(), grad_weights.data_ptr()
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).moe_combine_weighted_bwd, grad_out.data_ptr(), grad_code, eo, code,
                 row_of.data_ptr(), weights.data_ptr(), grad_expert_out.data_ptr(), gw, rows, tokens, top_k, hidden,
                 handle)
    if status:
        _fail(status, "moe_combine_weighted_bwd")


class MoeDispatch(torch.autograd.Function):
    """The tokens' rows in expert order: MoeDispatch.apply(x, row_of, slot_of). slot_of is moe_sort's
    first `rows` entries; rows past the last one are zeros."""

    @staticmethod
    def forward(ctx, x, row_of, slot_of):
        if row_of.shape[0] != x.shape[0]:          # the order of other tokens
            raise ValueError(f"row_of: expected {x.shape[0]} tokens as x has, got {row_of.shape[0]}")
        ctx.save_for_backward(row_of)
        ctx.tokens = x.shape[0]
        out = torch.empty((slot_of.shape[0], x.shape[1]), dtype=x.dtype, device=x.device)
        moe_dispatch_fwd(x.contiguous(), slot_of, row_of.shape[1], out)
        return out

    @staticmethod
    def backward(ctx, grad_out):
        binding._first_derivative_only("MoeDispatch", grad_out.requires_grad)
        row_of, = ctx.saved_tensors
        grad_x = torch.empty((ctx.tokens, grad_out.shape[1]), dtype=grad_out.dtype, device=grad_out.device)
        moe_dispatch_bwd(grad_out.contiguous(), row_of, grad_x)
        return grad_x, None, None


class MoeCombineWeighted(torch.autograd.Function):
    """The weighted sum of each token's rows: MoeCombineWeighted.apply(expert_out, row_of, weights,
    out_dtype=None). expert_out is kept for the backward pass only when weights need a gradient. The
    backward pass fills the rows' gradient with zeros before the kernel writes the rows that have a slot
    (65536 rows of 7168 bf16: 138 us beside 444)."""

    @staticmethod
    def forward(ctx, expert_out, row_of, weights, out_dtype=None):
        expert_out, weights = expert_out.contiguous(), weights.contiguous()
        ctx.save_for_backward(expert_out if ctx.needs_input_grad[2] else None, row_of, weights)
        ctx.rows, ctx.dtype = expert_out.shape[0], expert_out.dtype
        out = torch.empty((row_of.shape[0], expert_out.shape[1]), dtype=out_dtype or expert_out.dtype,
                          device=expert_out.device)
        moe_combine_weighted_fwd(expert_out, row_of, weights, out)
        return out

    @staticmethod
    def backward(ctx, grad_out):
        # each gradient is linear in grad_out and in the other input
        again = grad_out.requires_grad or (ctx.needs_input_grad[0] and ctx.needs_input_grad[2])
        binding._first_derivative_only("MoeCombineWeighted", again)
        expert_out, row_of, weights = ctx.saved_tensors
        # rows that belong to no slot have gradient 0
        grad_rows = torch.zeros((ctx.rows, grad_out.shape[1]), dtype=ctx.dtype, device=grad_out.device)
        grad_weights = torch.empty_like(weights) if ctx.needs_input_grad[2] else None
        moe_combine_weighted_bwd(grad_out.contiguous(), expert_out, row_of, weights, grad_rows, grad_weights)
        return grad_rows, None, grad_weights, None


# ---- 8-bit integers ---------------------------------------------------------------------

def quantize_rows_int8_fwd(x, q, scale, stream=None) -> None:
    """scale[r] = max|x[r]| / 127, q[r] = rint(127 x[r] / max|x[r]|). x [rows, cols] (bf16, fp16 or fp32);
    q int8 [rows, cols]; scale fp32 [rows]."""
    rows, cols = _matrix(x, "x")
    dev, code = x.get_device(), _code(x, "x")
    if not (dev >= 0 and x.is_contiguous()
            and q is not None and q.dtype is _I8 and q.get_device() == dev and q.shape == (rows, cols)
            and q.is_contiguous()
            and scale is not None and scale.dtype is _F32 and scale.get_device() == dev and scale.shape == (rows,)
            and scale.is_contiguous()):
        _refuse(dev, (x, "x", x.dtype, None), (q, "q", _I8, (rows, cols)), (scale, "scale", _F32, (rows,)))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).quantize_rows_int8_fwd, x.data_ptr(), code, q.data_ptr(), scale.data_ptr(), rows,
                 cols, handle)
    if status:
        _fail(status, "quantize_rows_int8_fwd")


def quantize_rows_int8(x):
    """(q, scale) of x in new tensors. x [..., cols]: the leading dimensions are rows, so that weights
    [experts, out, in] get a scale for each output channel."""
    q = torch.empty(x.shape, dtype=_I8, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=_F32, device=x.device)
    quantize_rows_int8_fwd(x.reshape(-1, x.shape[-1]).contiguous(), q.view(-1, x.shape[-1]), scale.view(-1))
    return q, scale


def grouped_gate_up_swiglu_int8_fwd(a, a_scale, slot_of, top_k: int, w_gate, w_gate_scale, w_up, w_up_scale, offs,
                                    probs, y, limit: float, stream=None) -> None:
    """gate_up grouped product in 8-bit integers + clamped SwiGLU x probs. a int8 [tokens, hidden] with
    a_scale fp32 [tokens]; slot_of int32 [rows] (row r reads token slot_of[r] // top_k) or None (row r
    reads row r of a, top_k 1); w_gate, w_up int8 [experts, inter, hidden] with scales fp32 [experts,
    inter]; offs int32 [experts] cumulative row counts (on the device); probs fp32 [rows] or None for 1;
    y bf16 [rows, inter]."""
    tokens, hidden = _matrix(a, "a")
    weight = experts, inter, _ = _experts(w_gate, "w_gate")
    rows, dev, channels = _matrix(y, "y")[0], a.get_device(), (experts, inter)
    if not (dev >= 0 and a.dtype is _I8 and a.is_contiguous()
            and a_scale is not None and a_scale.dtype is _F32 and a_scale.get_device() == dev
            and a_scale.shape == (tokens,) and a_scale.is_contiguous()
            and w_gate.dtype is _I8 and w_gate.get_device() == dev and weight[2] == hidden and w_gate.is_contiguous()
            and w_up is not None and w_up.dtype is _I8 and w_up.get_device() == dev and w_up.shape == weight
            and w_up.is_contiguous()
            and w_gate_scale is not None and w_gate_scale.dtype is _F32 and w_gate_scale.get_device() == dev
            and w_gate_scale.shape == channels and w_gate_scale.is_contiguous()
            and w_up_scale is not None and w_up_scale.dtype is _F32 and w_up_scale.get_device() == dev
            and w_up_scale.shape == channels and w_up_scale.is_contiguous()
            and offs is not None and offs.dtype is _I32 and offs.get_device() == dev and offs.shape == (experts,)
            and offs.is_contiguous()
            and y.dtype is _BF16 and y.get_device() == dev and y.shape == (rows, inter) and y.is_contiguous()):
        weight = (experts, inter, hidden)
        _refuse(dev, (a, "a", _I8, None), (a_scale, "a_scale", _F32, (tokens,)), (w_gate, "w_gate", _I8, weight),
                (w_gate_scale, "w_gate_scale", _F32, channels), (w_up, "w_up", _I8, weight),
                (w_up_scale, "w_up_scale", _F32, channels), (offs, "offs", _I32, (experts,)),
                (y, "y", _BF16, (rows, inter)))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).grouped_gate_up_swiglu_int8_fwd, a.data_ptr(), a_scale.data_ptr(),
                 _optional(slot_of, "slot_of", _I32, rows, dev), w_gate.data_ptr(), w_gate_scale.data_ptr(),
                 w_up.data_ptr(), w_up_scale.data_ptr(), offs.data_ptr(), _optional(probs, "probs", _F32, rows, dev),
                 y.data_ptr(), rows, tokens, top_k, hidden, inter, experts, limit, handle)
    if status:
        _fail(status, "grouped_gate_up_swiglu_int8_fwd")


def grouped_down_router_int8_fwd(h, h_scale, w_down, w_down_scale, offs, probs, out, stream=None) -> None:
    """Down grouped product in 8-bit integers + router multiply. h int8 [rows, inter] with h_scale fp32
    [rows]; w_down int8 [experts, hidden, inter] with w_down_scale fp32 [experts, hidden]; offs int32
    [experts] cumulative row counts (on the device); probs fp32 [rows] or None for 1; out [rows, hidden]
    bf16 or fp32."""
    rows, inter = _matrix(h, "h")
    weight = experts, hidden, _ = _experts(w_down, "w_down")
    dev = h.get_device()
    if out is None:
        _missing("out")
    if out.dtype is not _BF16 and out.dtype is not _F32:
        raise TypeError(f"out: expected bfloat16 or float32, got {out.dtype}")
    if not (dev >= 0 and h.dtype is _I8 and h.is_contiguous()
            and h_scale is not None and h_scale.dtype is _F32 and h_scale.get_device() == dev
            and h_scale.shape == (rows,) and h_scale.is_contiguous()
            and w_down.dtype is _I8 and w_down.get_device() == dev and weight[2] == inter and w_down.is_contiguous()
            and w_down_scale is not None and w_down_scale.dtype is _F32 and w_down_scale.get_device() == dev
            and w_down_scale.shape == (experts, hidden) and w_down_scale.is_contiguous()
            and offs is not None and offs.dtype is _I32 and offs.get_device() == dev and offs.shape == (experts,)
            and offs.is_contiguous()
            and out.get_device() == dev and out.shape == (rows, hidden) and out.is_contiguous()):
        _refuse(dev, (h, "h", _I8, None), (h_scale, "h_scale", _F32, (rows,)),
                (w_down, "w_down", _I8, (experts, hidden, inter)),
                (w_down_scale, "w_down_scale", _F32, (experts, hidden)), (offs, "offs", _I32, (experts,)),
                (out, "out", out.dtype, (rows, hidden)))
    handle = _raw_stream(dev) if stream is None else _handle(stream, dev)
    status = _on(dev, (_fns or _lib()).grouped_down_router_int8_fwd, h.data_ptr(), h_scale.data_ptr(),
                 w_down.data_ptr(), w_down_scale.data_ptr(), offs.data_ptr(),
                 _optional(probs, "probs", _F32, rows, dev), out.data_ptr(), DTYPE_CODE[out.dtype], rows, inter, hidden,
                 experts, handle)
    if status:
        _fail(status, "grouped_down_router_int8_fwd")
