"""The operators around the grouped (MoE) FP8 GEMMs: layer norm, routing,
token permutation and the gated activation with an 8-bit checkpoint (binding
over include/fp8mm_moe.h), their autograd ops, and the expert layer that runs
them together.

Functions named *_forward and *_backward are one call of the library each;
layer_norm, moe_route, moe_dispatch, moe_combine and fp8_swiglu are the same
operators as differentiable functions.  Matrices are 2-D and row-major with any
row stride, vectors, ids and weights dense (the differentiable functions make
their inputs so).  Errors are
those of the rest of the package: ValueError, NotImplementedError,
RuntimeError.
"""

import torch
from torch.autograd.function import once_differentiable

from . import (_ld, _lib, _need, _out_code, _ptr, fp8_grouped_linear_grad_weight, fp8_quantize_blockwise,
               fp8_quantize_grouped_128x1, fp8_quantize_grouped_dual, fp8_scaled_grouped_mm_v2)

__all__ = [
    "layer_norm_forward", "layer_norm_backward", "layer_norm", "moe_route_forward", "moe_route_backward", "moe_route",
    "moe_plan", "moe_dispatch_forward", "fp8_moe_dispatch", "moe_dispatch", "moe_combine_forward",
    "moe_combine_backward", "moe_combine", "fp8_swiglu_forward", "fp8_swiglu_backward", "fp8_swiglu", "FP8MoE",
    "fp8_moe",
]


# The current stream's handle without building a torch.cuda.Stream for it: 0.1
# against 2.0 us, of the 7 to 10 us that a call for a few tokens takes.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t):
    if _raw_stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _raw_stream(t.get_device())


def _rows(t, name):
    """Row stride of a 2-D tensor with unit column stride; its width where there
    is one row or none."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D row-major tensor")
    row, column = t.stride()
    if column != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be a 2-D row-major tensor")
    return row if shape[0] > 1 else shape[1]


def _need_float(t, name):
    """Element type of an activation: its C code."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype == torch.bfloat16:
        return _lib.OUT_BF16
    if t.dtype == torch.float32:
        return _lib.OUT_FP32
    raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")


def _like(t):
    """A dense tensor of t's shape and type (empty_like, where it is one, costs the host less)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _need_dense(t, dtype, shape, device, name):
    _need(t, dtype, name)
    if t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor on device {device}, got {list(t.shape)}")


def _code(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def _differentiates(*tensors):
    """Whether a gradient of one of the inputs can be asked for later.  (Inside an
    autograd function it is too late to ask: grad mode is off there, and its
    needs_input_grad is true of a parameter under no_grad too.)"""
    return torch.is_grad_enabled() and any(getattr(t, "requires_grad", False) for t in tensors)


# ------------------------------------------------------------------ layer norm

def _param(x, t, name):
    """Type code of a parameter vector of x's columns."""
    code = _need_float(t, name)
    if t.shape != x.shape[1:] or not t.is_contiguous() or t.get_device() != x.get_device():
        raise ValueError(f"{name} must be a contiguous [{x.shape[1]}] tensor on {x.device}, got {list(t.shape)}")
    return code


def _params(x, weight, bias):
    """Type code of the parameters, which are of one type."""
    if weight is None:
        return _lib.OUT_FP32 if bias is None else _param(x, bias, "bias")
    code = _param(x, weight, "weight")
    if bias is not None and _param(x, bias, "bias") != code:
        raise ValueError("weight and bias must have the same dtype")
    return code


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5):
    """x [R, C] bf16 or fp32 -> (y like x, mean float32 [R], rstd float32 [R]):
    y = (x - mean) rstd weight + bias.  weight and bias: [C], bf16 or fp32."""
    dtype = _need_float(x, "x")
    ld = _rows(x, "x")
    params = _params(x, weight, bias)
    R, C = x.shape
    y = _like(x)
    mean, rstd = x.new_empty((2, R), dtype=torch.float32).unbind(0)
    st = _lib.load().fp8mm_layer_norm(x.data_ptr(), dtype, R, C, ld, _ptr(weight), _ptr(bias), params, eps,
                                      y.data_ptr(), C, mean.data_ptr(), rstd.data_ptr(), _stream(x))
    _lib.check(st, "fp8mm_layer_norm")
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, need_dx=True, need_params=True, param_dtype=None):
    """(dx, dweight, dbias) of layer_norm_forward from its x, weight, mean and
    rstd.  dweight and dbias have the weight's type (param_dtype, or float32,
    where there is no weight); None where not needed."""
    dtype = _need_float(x, "x")
    if _need_float(dy, "dy") != dtype or dy.shape != x.shape or dy.get_device() != x.get_device():
        raise ValueError("dy must have the dtype, shape and device of x")
    ld_dy, ld_x = _rows(dy, "dy"), _rows(x, "x")
    R, C = x.shape
    _params(x, weight, None)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _need_dense(t, torch.float32, (R,), x.get_device(), name)
    if weight is not None:
        param_dtype = weight.dtype
    elif param_dtype is None:
        param_dtype = torch.float32
    lib = _lib.load()
    dx = _like(x) if need_dx else None
    dweight = dbias = workspace = None
    size = 0
    if need_params:
        dweight = x.new_empty((C,), dtype=param_dtype)
        dbias = torch.empty_like(dweight)
        size = lib.fp8mm_layer_norm_backward_workspace(R, C)
        if size > 0:
            workspace = x.new_empty((size,), dtype=torch.uint8)
    st = lib.fp8mm_layer_norm_backward(dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, dtype, R, C, _ptr(weight),
                                       _out_code(param_dtype), mean.data_ptr(), rstd.data_ptr(), _ptr(dx), C,
                                       _ptr(dweight), _ptr(dbias), _ptr(workspace), size, _stream(x))
    _lib.check(st, "fp8mm_layer_norm_backward")
    return dx, dweight, dbias


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        flat = x.contiguous().view(-1, x.shape[-1])
        weight = None if weight is None else weight.contiguous()
        bias = None if bias is None else bias.contiguous()
        y, mean, rstd = layer_norm_forward(flat, weight, bias, eps)
        ctx.save_for_backward(flat, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dweight, dbias = layer_norm_backward(dy.to(x.dtype).contiguous().view(x.shape), x, weight, mean, rstd,
                                                 need[0], need[1] or need[2], ctx.bias_dtype)
        return (dx.view(dy.shape) if need[0] else None, dweight if need[1] else None, dbias if need[2] else None, None)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over the last dimension of x (any leading dimensions),
    differentiable in x, weight and bias."""
    return _LayerNorm.apply(x, weight, bias, eps)


# --------------------------------------------------------------------- routing

def moe_route_forward(logits, k, score="softmax", bias=None, groups=1, group_topk=None, group_score="max",
                      renormalize=True, scale=1.0):
    """logits [T, E] bf16 or fp32 -> (ids int32 [T, k], weights float32 [T, k]).

    Scores are the softmax or sigmoid of a token's logits; the k experts with
    the largest score + bias (float32 [E]) are chosen, in descending order,
    ties to the lower index, after keeping the group_topk best of `groups`
    equal runs of experts (by their best, or the sum of their two best:
    group_score "max" or "top2").  Weights are the chosen scores, divided by
    their sum if renormalize, times scale.  Experts with a logit or bias of
    -inf are never chosen; slots without an expert get id -1 and weight 0."""
    dtype = _need_float(logits, "logits")
    ld = _rows(logits, "logits")
    T, E = logits.shape
    if bias is not None:
        _need_dense(bias, torch.float32, (E,), logits.get_device(), "bias")
    k = int(k)
    slots = max(k, 0)
    ids = logits.new_empty((T, slots), dtype=torch.int32)
    weights = logits.new_empty((T, slots), dtype=torch.float32)
    st = _lib.load().fp8mm_moe_route(logits.data_ptr(), dtype, T, E, ld, _ptr(bias),
                                     _code(_lib.SCORES, score, "score"), k, groups,
                                     groups if group_topk is None else group_topk,
                                     _code(_lib.GROUP_SCORES, group_score, "group_score"), 1 if renormalize else 0,
                                     scale, ids.data_ptr(), weights.data_ptr(), _stream(logits))
    _lib.check(st, "fp8mm_moe_route")
    return ids, weights


def moe_route_backward(grad_weights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """Gradient of the logits (their type and shape) from the gradient of
    moe_route_forward's weights, the chosen ids (different ones in a token, as
    the forward gives them) held fixed."""
    dtype = _need_float(logits, "logits")
    ld = _rows(logits, "logits")
    T, E = logits.shape
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}, k], got {list(ids.shape)}")
    _need_dense(ids, torch.int32, ids.shape, logits.get_device(), "ids")
    _need_dense(grad_weights, torch.float32, ids.shape, logits.get_device(), "grad_weights")
    grad = _like(logits)
    st = _lib.load().fp8mm_moe_route_backward(grad_weights.data_ptr(), logits.data_ptr(), dtype, T, E, ld,
                                              ids.data_ptr(), ids.shape[1], _code(_lib.SCORES, score, "score"),
                                              1 if renormalize else 0, scale, grad.data_ptr(), E, _stream(logits))
    _lib.check(st, "fp8mm_moe_route_backward")
    return grad


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, bias, groups, group_topk, group_score, renormalize, scale):
        logits = logits.contiguous()
        bias = None if bias is None else bias.contiguous()
        ids, weights = moe_route_forward(logits, k, score, bias, groups, group_topk, group_score, renormalize, scale)
        ctx.save_for_backward(logits, ids)
        ctx.args = score, renormalize, scale
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, grad_weights):
        logits, ids = ctx.saved_tensors
        grad = moe_route_backward(grad_weights.contiguous(), logits, ids, *ctx.args)
        return grad, None, None, None, None, None, None, None, None


def moe_route(logits, k, score="softmax", bias=None, groups=1, group_topk=None, group_score="max", renormalize=True,
              scale=1.0):
    """moe_route_forward, differentiable in the logits through the weights."""
    return _Route.apply(logits, k, score, bias, groups, group_topk, group_score, renormalize, scale)


# ----------------------------------------------------------------- permutation

def moe_plan(ids, experts):
    """ids int32 [T, k] -> (offsets int32 [experts], row_of_slot int32 [T, k]):
    the experts' cumulative end rows for the grouped calls, and each slot's row
    by a stable sort by expert.  Slots with an id outside [0, experts) take the
    rows past offsets[-1] and are written as ~row (negative)."""
    _need(ids, torch.int32, "ids")
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous [T, k] tensor")
    T, k = ids.shape
    lib = _lib.load()
    size = lib.fp8mm_moe_plan_workspace(T, k, experts)
    workspace = ids.new_empty((size,), dtype=torch.uint8) if size > 0 else None
    offsets = ids.new_empty((max(int(experts), 0),))
    row_of_slot = torch.empty_like(ids)
    st = lib.fp8mm_moe_plan(ids.data_ptr(), T, k, experts, offsets.data_ptr(), row_of_slot.data_ptr(), _ptr(workspace),
                            max(size, 0), _stream(ids))
    _lib.check(st, "fp8mm_moe_plan")
    return offsets, row_of_slot


def _need_slots(row_of_slot, tokens, device):
    _need(row_of_slot, torch.int32, "row_of_slot")
    if (row_of_slot.dim() != 2 or (tokens is not None and row_of_slot.shape[0] != tokens) or
            not row_of_slot.is_contiguous() or row_of_slot.get_device() != device):
        raise ValueError("row_of_slot must be a contiguous [T, k] tensor on the rows' device")
    return row_of_slot.shape


def moe_dispatch_forward(x, row_of_slot):
    """x [T, C] bf16 or fp32 -> rows [T k, C] in expert order (zeros in the rows
    of slots without an expert)."""
    dtype = _need_float(x, "x")
    ld = _rows(x, "x")
    T, k = _need_slots(row_of_slot, x.shape[0], x.get_device())
    C = x.shape[1]
    out = x.new_empty((T * k, C))
    st = _lib.load().fp8mm_moe_dispatch(x.data_ptr(), dtype, T, C, ld, row_of_slot.data_ptr(), k, out.data_ptr(), C,
                                        _stream(x))
    _lib.check(st, "fp8mm_moe_dispatch")
    return out


def fp8_moe_dispatch(x, row_of_slot):
    """x bf16 [T, C] -> (codes uint8 [T k, C], scales float32 [C/128, T k]) in
    expert order: the 1x128 quantization of the dispatched rows, each token
    quantized once.  Rows of slots without an expert: codes 0, scales 1."""
    _need(x, torch.bfloat16, "x")
    ld = _ld(x, "x")
    T, k = _need_slots(row_of_slot, x.shape[0], x.get_device())
    C = x.shape[1]
    q = x.new_empty((T * k, C), dtype=torch.uint8)
    scale = x.new_empty((C // 128, T * k), dtype=torch.float32)
    st = _lib.load().fp8_moe_dispatch(x.data_ptr(), T, C, ld, row_of_slot.data_ptr(), k, q.data_ptr(), C,
                                      scale.data_ptr(), _stream(x))
    _lib.check(st, "fp8_moe_dispatch")
    return q, scale


def moe_combine_forward(rows, row_of_slot, weights=None):
    """rows [T k, C] in expert order -> [T, C]: each token's rows, weighted
    (float32 [T, k]; None: 1) and added in slot order."""
    dtype = _need_float(rows, "rows")
    ld = _rows(rows, "rows")
    T, k = _need_slots(row_of_slot, None, rows.get_device())
    if rows.shape[0] != T * k:
        raise ValueError(f"rows must have T k = {T * k} rows, got {rows.shape[0]}")
    if weights is not None:
        _need_dense(weights, torch.float32, (T, k), rows.get_device(), "weights")
    C = rows.shape[1]
    out = rows.new_empty((T, C))
    st = _lib.load().fp8mm_moe_combine(rows.data_ptr(), dtype, T, C, ld, row_of_slot.data_ptr(), _ptr(weights), k,
                                       out.data_ptr(), C, _stream(rows))
    _lib.check(st, "fp8mm_moe_combine")
    return out


def moe_combine_backward(grad_out, rows, row_of_slot, weights=None, need_rows=True, need_weights=True):
    """(grad_rows [T k, C], grad_weights float32 [T, k]) of moe_combine_forward;
    None where not needed.  rows may be None without need_weights."""
    dtype = _need_float(grad_out, "grad_out")
    ld_go = _rows(grad_out, "grad_out")
    T, k = _need_slots(row_of_slot, grad_out.shape[0], grad_out.get_device())
    C = grad_out.shape[1]
    ld = 0
    if rows is not None:
        if (_need_float(rows, "rows") != dtype or rows.shape != (T * k, C) or
                rows.get_device() != grad_out.get_device()):
            raise ValueError(f"rows must be [{T * k}, {C}] of grad_out's dtype and device")
        ld = _rows(rows, "rows")
    elif need_weights:
        raise ValueError("rows are needed for the gradient of the weights")
    if weights is not None:
        _need_dense(weights, torch.float32, (T, k), grad_out.get_device(), "weights")
    grad_rows = grad_out.new_empty((T * k, C)) if need_rows else None
    grad_weights = grad_out.new_empty((T, k), dtype=torch.float32) if need_weights else None
    st = _lib.load().fp8mm_moe_combine_backward(grad_out.data_ptr(), ld_go, _ptr(rows), ld, dtype, T, C,
                                                row_of_slot.data_ptr(), _ptr(weights), k, _ptr(grad_rows), C,
                                                _ptr(grad_weights), _stream(grad_out))
    _lib.check(st, "fp8mm_moe_combine_backward")
    return grad_rows, grad_weights


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_of_slot):
        row_of_slot = row_of_slot.contiguous()
        ctx.save_for_backward(row_of_slot)
        return moe_dispatch_forward(x.contiguous(), row_of_slot)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        row_of_slot, = ctx.saved_tensors
        return moe_combine_forward(grad.contiguous(), row_of_slot), None


def moe_dispatch(x, row_of_slot):
    """moe_dispatch_forward, differentiable in x."""
    return _Dispatch.apply(x, row_of_slot)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, row_of_slot, weights):
        rows, row_of_slot = rows.contiguous(), row_of_slot.contiguous()
        weights = None if weights is None else weights.contiguous()
        # the rows are for the gradient of the weights alone
        ctx.save_for_backward(rows if ctx.needs_input_grad[2] else None, row_of_slot, weights)
        ctx.dtype = rows.dtype
        return moe_combine_forward(rows, row_of_slot, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        rows, row_of_slot, weights = ctx.saved_tensors
        need = ctx.needs_input_grad
        grad_rows, grad_weights = moe_combine_backward(grad.to(ctx.dtype).contiguous(), rows, row_of_slot, weights,
                                                       need[0], need[2])
        return grad_rows, None, grad_weights


def moe_combine(rows, row_of_slot, weights=None):
    """moe_combine_forward, differentiable in rows and weights."""
    return _Combine.apply(rows, row_of_slot, weights)


# ------------------------------------------------------------ gated activation

def fp8_swiglu_forward(x, out="bf16", checkpoint=True):
    """x = [gate, up] bf16 [R, 2 F], F % 128 == 0 -> (h, checkpoint) with h =
    silu(gate) up.

    out "bf16": h is bf16 [R, F]; "fp8": h is the pair (codes uint8 [R, F],
    scales float32 [F/128, R]) of its 1x128 quantization.  checkpoint: the pair
    (codes uint8 [R, 2 F], scales float32 [2F/128, R]) of x's 1x128
    quantization, what fp8_swiglu_backward needs; None if not wanted."""
    _need(x, torch.bfloat16, "x")
    ld = _ld(x, "x")
    if out not in ("bf16", "fp8"):
        raise ValueError(f"out must be 'bf16' or 'fp8', got {out!r}")
    R, F2 = x.shape
    if F2 % 256:
        raise ValueError(f"x must have a multiple of 256 columns (gate and up of 128 each), got {F2}")
    F = F2 // 2
    h = q = s = c = cs = None
    if out == "bf16":
        h = x.new_empty((R, F), dtype=torch.bfloat16)
    else:
        q = x.new_empty((R, F), dtype=torch.uint8)
        s = x.new_empty((F // 128, R), dtype=torch.float32)
    if checkpoint:
        c = x.new_empty((R, F2), dtype=torch.uint8)
        cs = x.new_empty((F2 // 128, R), dtype=torch.float32)
    st = _lib.load().fp8_swiglu(x.data_ptr(), R, F, ld, _ptr(h), F, _ptr(q), F, _ptr(s), _ptr(c), F2, _ptr(cs),
                                _stream(x))
    _lib.check(st, "fp8_swiglu")
    return (h if out == "bf16" else (q, s)), ((c, cs) if checkpoint else None)


def fp8_swiglu_backward(grad_h, codes, scale, recompute=False):
    """(grad_x bf16 [R, 2 F], h) from grad_h bf16 [R, F] and the checkpoint of
    fp8_swiglu_forward; h is the activation again, bf16 [R, F], if recompute
    (for the weight gradient of the product that reads it), else None."""
    _need(grad_h, torch.bfloat16, "grad_h")
    ld = _ld(grad_h, "grad_h")
    R, F = grad_h.shape
    if F % 128:
        raise ValueError(f"grad_h must have a multiple of 128 columns, got {F}")
    _need_dense(codes, torch.uint8, (R, 2 * F), grad_h.get_device(), "codes")
    _need_dense(scale, torch.float32, (2 * F // 128, R), grad_h.get_device(), "scale")
    grad_x = grad_h.new_empty((R, 2 * F), dtype=torch.bfloat16)
    h = grad_h.new_empty((R, F), dtype=torch.bfloat16) if recompute else None
    st = _lib.load().fp8_swiglu_backward(grad_h.data_ptr(), ld, codes.data_ptr(), 2 * F, scale.data_ptr(), R, F,
                                         grad_x.data_ptr(), 2 * F, _ptr(h), F, _stream(grad_h))
    _lib.check(st, "fp8_swiglu_backward")
    return grad_x, h


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x):
        h, checkpoint = fp8_swiglu_forward(x.contiguous(), "bf16", ctx.needs_input_grad[0])
        if checkpoint is not None:
            ctx.save_for_backward(*checkpoint)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_h):
        return fp8_swiglu_backward(grad_h.to(torch.bfloat16).contiguous(), *ctx.saved_tensors)[0]


def fp8_swiglu(x):
    """silu(gate) up of x = [gate, up] bf16 [R, 2 F], differentiable; the
    backward pass reads x in 8 bits (1x128 codes), and x itself is not kept.
    The codes are made only where a gradient can follow."""
    if _differentiates(x):
        return _Swiglu.apply(x)
    return fp8_swiglu_forward(x.contiguous(), "bf16", False)[0]


# ---------------------------------------------------------------- expert layer

def _weight_codes(w):
    """[E, N, K] bf16 -> 128x128 codes of the same shape and scales per expert."""
    E, N, K = w.shape
    q, s = fp8_quantize_blockwise(w.contiguous().view(E * N, K), (128, 128))
    return q.view(E, N, K), s.view(E, N // 128, K // 128)


def _experts_mm(q, s, w_q, w_s, offsets, layout="NK"):
    """The grouped product of expert-order rows in the blockwise recipe.  Rows of
    slots without an expert are left unwritten: nothing that follows lets them
    into a row that has one (combine and the per-expert quantizers skip them)."""
    N = w_q.shape[1 if layout == "NK" else 2]
    out = q.new_empty((q.shape[0], N), dtype=torch.bfloat16)
    return fp8_scaled_grouped_mm_v2(q, w_q, offsets, s, "1x128", w_s, "128x128", b_layout=layout, out=out)


def _experts_forward(x, w_in, w_out, ids, weights, train, train_weights):
    """(y, what FP8MoE.backward needs: nothing without train, no rows without
    train_weights)."""
    for t, name in ((x, "x"), (w_in, "w_in"), (w_out, "w_out")):
        _need(t, torch.bfloat16, name)
    E = w_in.shape[0]
    if w_in.dim() != 3 or w_out.dim() != 3 or w_in.shape != (E, 2 * w_out.shape[2], w_out.shape[1]):
        raise ValueError("w_in must be [E, 2 F, C] and w_out [E, C, F], "
                         f"got {list(w_in.shape)} and {list(w_out.shape)}")
    if w_out.shape[0] != E:
        raise ValueError(f"w_in has {E} experts, w_out {w_out.shape[0]}")
    x, weights = x.contiguous(), weights.contiguous()
    offsets, row_of_slot = moe_plan(ids.contiguous(), E)
    q_in, s_in = _weight_codes(w_in)
    q_out, s_out = _weight_codes(w_out)
    q, s = fp8_moe_dispatch(x, row_of_slot)
    gate_up = _experts_mm(q, s, q_in, s_in, offsets)
    (hq, hs), checkpoint = fp8_swiglu_forward(gate_up, "fp8", train)
    rows = _experts_mm(hq, hs, q_out, s_out, offsets)
    y = moe_combine_forward(rows, row_of_slot, weights)
    if not train:
        return y, ()
    return y, (x, q_in, s_in, q_out, s_out, *checkpoint, rows if train_weights else None, offsets, row_of_slot, weights)


class FP8MoE(torch.autograd.Function):
    """The experts of a mixture-of-experts block on routed tokens,

      y[t] = sum_j weights[t, j] down_e(silu(gate) up), [gate, up] = w_in_e x[t],
      e = ids[t, j]

    in the blockwise FP8 recipe.  x [T, C], w_in [E, 2 F, C], w_out [E, C, F]
    bf16, ids int32 [T, k] and weights float32 [T, k] from moe_route; C and F
    multiples of 128.

      forward:  plan; dispatch x as 1x128 codes; grouped GEMM; gated activation
                to 1x128 codes and the 8-bit checkpoint; grouped GEMM; combine
      backward: combine's; the second product's two gradients (its input again
                from the checkpoint); the activation's from the checkpoint; the
                first product's two gradients; dispatch's

    Kept for the backward: x once per token, the checkpoint (2 F bytes a row in
    place of 4 F), the weights' codes and, where `weights` needs its gradient, the
    rows before combine."""

    @staticmethod
    def forward(ctx, x, w_in, w_out, ids, weights):
        y, saved = _experts_forward(x, w_in, w_out, ids, weights, any(ctx.needs_input_grad),
                                    ctx.needs_input_grad[4])
        ctx.save_for_backward(*saved)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, q_in, s_in, q_out, s_out, codes, scale, rows, offsets, row_of_slot, weights = ctx.saved_tensors
        need_x, need_in, need_out, _, need_w = ctx.needs_input_grad
        g = grad_out.to(torch.bfloat16).contiguous()
        M = row_of_slot.numel()
        grad_x = grad_in = grad_w_out = None
        grad_rows, grad_weights = moe_combine_backward(g, rows, row_of_slot, weights, need_x or need_in or need_out,
                                                       need_w)
        if need_x or need_in or need_out:
            if need_out:
                qg, sg, qgt, sgt = fp8_quantize_grouped_dual(grad_rows, offsets)
            else:
                qg, sg = fp8_quantize_blockwise(grad_rows, (1, 128))
            grad_h = _experts_mm(qg, sg, q_out, s_out, offsets, "KN")
            grad_gate_up, h = fp8_swiglu_backward(grad_h, codes, scale, recompute=need_out)
            if need_out:
                qht, sht = fp8_quantize_grouped_128x1(h, offsets)
                grad_w_out = fp8_grouped_linear_grad_weight(qgt, sgt, qht, sht, offsets, M)
            if need_in:
                qg, sg, qgt, sgt = fp8_quantize_grouped_dual(grad_gate_up, offsets)
                qxt, sxt = fp8_quantize_grouped_128x1(moe_dispatch_forward(x, row_of_slot), offsets)
                grad_in = fp8_grouped_linear_grad_weight(qgt, sgt, qxt, sxt, offsets, M)
            elif need_x:
                qg, sg = fp8_quantize_blockwise(grad_gate_up, (1, 128))
            if need_x:
                grad_rows = _experts_mm(qg, sg, q_in, s_in, offsets, "KN")
                grad_x = moe_combine_forward(grad_rows, row_of_slot)
        return grad_x, grad_in, grad_w_out, None, grad_weights


def fp8_moe(x, w_in, w_out, ids, weights):
    """The expert layer through FP8MoE (differentiable in x, w_in, w_out and
    weights; ids and weights from moe_route).  Where no gradient can follow (no_grad,
    or no input that needs one), its forward alone, without the 8-bit checkpoint."""
    if _differentiates(x, w_in, w_out, weights):
        return FP8MoE.apply(x, w_in, w_out, ids, weights)
    return _experts_forward(x, w_in, w_out, ids, weights, False, False)[0]
