"""The operators around a block's dense FP8 products and its router: the RMS norm
that adds the residual and gives the product's codes, the balance loss with the
experts' counts, and low-rank adapters of many requests beside a shared projection
(binding over include/fp8mm_block.h), and their autograd ops.

Functions named *_forward and *_backward are one call of the library each; rms_norm,
moe_balance_loss and lora are the same operators as differentiable functions.
Matrices are 2-D and row-major with any row stride, vectors, panels, ids and ends
dense (the differentiable functions make their inputs so).  Kernels go to the
current stream of the tensors' device, which need not be the current device.  Errors
are those of the rest of the package: ValueError, NotImplementedError, RuntimeError.
"""

import torch
from torch.autograd.function import once_differentiable

from . import _lib, _need, _out_code, _ptr, _recipe
from .moe import _code, _differentiates, _like, _need_dense, _need_float, _rows, _stream

__all__ = [
    "rms_norm_forward", "fp8_rms_norm_forward", "rms_norm_backward", "rms_norm", "moe_balance_loss_forward",
    "moe_balance_loss_backward", "moe_balance_loss", "lora_forward", "lora_backward", "lora",
]


# The current device's number, without the checks around torch.cuda.current_device (0.14
# against 0.26 us).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, t, *args):
    """The library's call on the current stream of t's device."""
    fn = getattr(_lib._lib or _lib.load(), name)
    if t.get_device() == _current_device():
        st = fn(*args, _stream(t))
    else:
        with torch.cuda.device(t.get_device()):
            st = fn(*args, _stream(t))
    if st != _lib.OK:
        _lib.check(st, name)


# The checks below first ask whether all is well, in a few attribute reads, and look for
# what is wrong only if not: the calls for a few tokens take the host longer than the
# GPU, and 2 to 3 of their 10 to 13 us were checks.

def _dense(t, dtype, shape, device, name):
    """t is a dense tensor of this type, shape and device number."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    _need_dense(t, dtype, shape, device, name)


_CODES = {torch.bfloat16: _lib.OUT_BF16, torch.float32: _lib.OUT_FP32}


def _matrix(t, name):
    """(type code, row stride, device number) of a bf16 or float32 matrix."""
    try:
        device, code = t.get_device(), _CODES[t.dtype]
        R, C = t.shape
        row, column = t.stride()
        if device >= 0 and (column == 1 or C <= 1):
            return code, (row if R > 1 else C), device
    except (AttributeError, KeyError, ValueError):
        pass
    return _need_float(t, name), _rows(t, name), t.get_device()


def _need_like(t, x, name):
    """Row stride of a matrix of x's type, shape and device."""
    if not isinstance(t, torch.Tensor) or t.dtype != x.dtype or t.shape != x.shape or t.get_device() != x.get_device():
        raise ValueError(f"{name} must be a {list(x.shape)} tensor of {x.dtype} on {x.device}")
    return _rows(t, name)


# -------------------------------------------------------------------- RMS norm

def _weight(x, weight):
    """Type code of the weight vector."""
    if weight is None:
        return _lib.OUT_FP32
    try:
        if weight.shape == x.shape[1:] and weight.get_device() == x.get_device() and weight.is_contiguous():
            return _CODES[weight.dtype]
    except (AttributeError, KeyError):
        pass
    code = _need_float(weight, "weight")
    if weight.shape != x.shape[1:] or not weight.is_contiguous() or weight.get_device() != x.get_device():
        raise ValueError(f"weight must be a contiguous [{x.shape[1]}] tensor on {x.device}, got {list(weight.shape)}")
    return code


def _rms(x, weight, residual, eps, recipe, want_y):
    dtype, ld, _ = _matrix(x, "x")
    params = _weight(x, weight)
    R, C = x.shape
    h, ld_res = x, 0
    if residual is not None:
        ld_res = _need_like(residual, x, "residual")
        h = _like(x)
    q = scale = None
    code = _lib.RECIPES["1x128"]
    if recipe is not None:
        code = _recipe(recipe)
        q = x.new_empty((R, C), dtype=torch.uint8)
        scale = x.new_empty((R, 1) if code == _lib.RECIPES["rowwise"] else (C // 128, R), dtype=torch.float32)
    y = _like(x) if want_y else None
    rstd = x.new_empty((R,), dtype=torch.float32)
    _call("fp8mm_rms_norm", x, x.data_ptr(), ld, _ptr(residual), ld_res, dtype, R, C, _ptr(weight), params, eps,
          h.data_ptr() if residual is not None else None, C, _ptr(y), C, _ptr(q), C, _ptr(scale), code,
          rstd.data_ptr())
    return q, scale, y, h, rstd


def rms_norm_forward(x, weight=None, residual=None, eps=1e-6):
    """x [R, C] bf16 or fp32 -> (y like x, h like x, rstd float32 [R]): h = x +
    residual rounded to x's type (x itself without one), y = h rstd weight with
    rstd = 1 / sqrt(mean(h^2) + eps).  weight: [C], bf16 or fp32."""
    return _rms(x, weight, residual, eps, None, True)[2:]


def fp8_rms_norm_forward(x, weight=None, residual=None, eps=1e-6, recipe="1x128", y=False):
    """x bf16 [R, C] -> (codes uint8 [R, C], scale, y, h, rstd): rms_norm_forward with
    the codes and scales of y's float32 values, as the product that follows takes
    them: recipe "1x128" (scale float32 [C/128, R]; C a multiple of 128) or "rowwise"
    ([R, 1], with the epsilon; C a multiple of 16).  y itself (bf16) if asked for,
    else None."""
    _need(x, torch.bfloat16, "x")
    if x.dim() != 2:
        raise ValueError("x must be a 2-D row-major tensor")
    return _rms(x, weight, residual, eps, recipe, y)


def rms_norm_backward(dy, h, weight, rstd, grad_h=None, need_dx=True, need_weight=True, param_dtype=None):
    """(dx, dweight) of rms_norm_forward from its h, weight and rstd.  dx is the
    gradient of x and of the residual; grad_h, the gradient that arrives at h from
    behind, is added to it.  dweight has the weight's type (param_dtype, or float32,
    where there is no weight); None where not needed."""
    dtype, ld_h, device = _matrix(h, "h")
    ld_dy = _need_like(dy, h, "dy")
    ld_gh = 0 if grad_h is None else _need_like(grad_h, h, "grad_h")
    R, C = h.shape
    params = _weight(h, weight)
    _dense(rstd, torch.float32, (R,), device, "rstd")
    if weight is None:
        param_dtype = torch.float32 if param_dtype is None else param_dtype
        params = _out_code(param_dtype)
    else:
        param_dtype = weight.dtype
    dx = _like(h) if need_dx else None
    dweight = workspace = None
    size = 0
    if need_weight:
        dweight = h.new_empty((C,), dtype=param_dtype)
        size = _lib.load().fp8mm_rms_norm_backward_workspace(R, C)
        if size > 0:
            workspace = h.new_empty((size,), dtype=torch.uint8)
    _call("fp8mm_rms_norm_backward", h, dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, _ptr(grad_h), ld_gh, dtype, R, C,
          _ptr(weight), params, rstd.data_ptr(), _ptr(dx), C, _ptr(dweight), _ptr(workspace), size)
    return dx, dweight


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        flat = x.contiguous().view(-1, x.shape[-1])
        weight = None if weight is None else weight.contiguous()
        if residual is not None:
            residual = residual.contiguous().view(flat.shape)
        y, h, rstd = rms_norm_forward(flat, weight, residual, eps)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, weight, rstd)
        y = y.view(x.shape)
        return y if residual is None else (y, h.view(x.shape))

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, grad_h=None):
        h, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None:                           # the residual stream alone was used
            return grad_h, torch.zeros_like(weight) if need[1] else None, grad_h if need[2] else None, None
        shape = dy.shape
        dy = dy.to(h.dtype).contiguous().view(h.shape)
        if grad_h is not None:
            grad_h = grad_h.to(h.dtype).contiguous().view(h.shape)
        dx, dweight = rms_norm_backward(dy, h, weight, rstd, grad_h, need[0] or need[2], need[1])
        if dx is not None:
            dx = dx.view(shape)
        return dx if need[0] else None, dweight, dx if need[2] else None, None


def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """RMS norm over the last dimension of x (any leading dimensions),
    differentiable in x, weight and residual: y, or with a residual (y, h), h = x +
    residual being the next residual."""
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual must have the shape and dtype of x")
    return _RmsNorm.apply(x, weight, residual, eps)


# ---------------------------------------------------------------- balance loss

def _sequences(ends, logits):
    if ends is None:
        return 1
    _need(ends, torch.int32, "ends")
    if ends.dim() != 1 or ends.numel() < 1 or not ends.is_contiguous() or ends.get_device() != logits.get_device():
        raise ValueError("ends must be a contiguous int32 [S] tensor of at least one sequence on the logits' device")
    return ends.numel()


def moe_balance_loss_forward(logits, ids, score="softmax", coeff=1.0, ends=None):
    """logits [T, E] bf16 or fp32 and the chosen ids int32 [T, k] (-1: an empty slot) ->
    (loss float32 [], counts int32 [S, E], tokens int32 [S]).

    ends: int32 [S], the sequences' ascending end rows; rows behind the last belong to
    none.  None: one sequence of all rows.  A row of -inf alone is padding and does not
    count.  With p = softmax(logits), or the sigmoids divided by their sum, and n the
    tokens of a sequence, its loss is coeff sum_e (E counts_e / (k n)) (sum_t p_te /
    n); loss is the mean over the sequences that have tokens."""
    dtype, ld, device = _matrix(logits, "logits")
    T, E = logits.shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError(f"ids must be an int32 [{T}, k] tensor")
    _dense(ids, torch.int32, (T, ids.shape[1]), device, "ids")
    S = _sequences(ends, logits)
    size = _lib.load().fp8mm_moe_balance_loss_workspace(T, E, S)
    loss = logits.new_empty((), dtype=torch.float32)
    counts = ids.new_empty((S, E))
    tokens = ids.new_empty((S,))
    workspace = logits.new_empty((size,), dtype=torch.uint8) if size > 0 else None
    _call("fp8mm_moe_balance_loss", logits, logits.data_ptr(), dtype, T, E, ld, ids.data_ptr(), ids.shape[1],
          _code(_lib.SCORES, score, "score"), _ptr(ends), S, coeff, loss.data_ptr(), counts.data_ptr(),
          tokens.data_ptr(), _ptr(workspace), max(size, 0))
    return loss, counts, tokens


def moe_balance_loss_backward(grad_loss, logits, counts, tokens, k, score="softmax", coeff=1.0, ends=None):
    """Gradient of the logits (their type and shape) from the gradient of
    moe_balance_loss_forward's loss (float32 []), its counts and tokens; k: slots of a
    token.  Zeros in rows of no sequence and in padding."""
    dtype, ld, device = _matrix(logits, "logits")
    T, E = logits.shape
    S = _sequences(ends, logits)
    _need(grad_loss, torch.float32, "grad_loss")
    if grad_loss.numel() != 1 or grad_loss.get_device() != device:
        raise ValueError("grad_loss must be one float32 number on the logits' device")
    _dense(counts, torch.int32, (S, E), device, "counts")
    _dense(tokens, torch.int32, (S,), device, "tokens")
    grad = _like(logits)
    _call("fp8mm_moe_balance_loss_backward", logits, grad_loss.data_ptr(), logits.data_ptr(), dtype, T, E, ld,
          counts.data_ptr(), tokens.data_ptr(), k, _code(_lib.SCORES, score, "score"), _ptr(ends), S, coeff,
          grad.data_ptr(), E)
    return grad


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, score, coeff, ends):
        logits, ids = logits.contiguous(), ids.contiguous()
        ends = None if ends is None else ends.contiguous()
        loss, counts, tokens = moe_balance_loss_forward(logits, ids, score, coeff, ends)
        ctx.save_for_backward(logits, counts, tokens, ends)
        ctx.args = ids.shape[1], score, coeff
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, _):
        logits, counts, tokens, ends = ctx.saved_tensors
        grad = moe_balance_loss_backward(grad_loss.float(), logits, counts, tokens, *ctx.args, ends)
        return grad, None, None, None, None


def moe_balance_loss(logits, ids, score="softmax", coeff=1.0, ends=None):
    """(loss, counts) of moe_balance_loss_forward, the loss differentiable in the
    logits (the choice itself has no gradient)."""
    return _BalanceLoss.apply(logits, ids, score, coeff, ends)


# -------------------------------------------------------------------- adapters

def _panels(down, up, T, ids, scales, device):
    """(K, n, r, N) of an adapter call for T tokens on a device."""
    try:
        n, r, K = down.shape
        N = up.shape[2]
    except (AttributeError, ValueError, IndexError):
        raise ValueError("down and up must be [adapters, rank, columns] tensors") from None
    _dense(down, torch.bfloat16, (n, r, K), device, "down")
    _dense(up, torch.bfloat16, (n, r, N), device, "up")
    _dense(ids, torch.int32, (T,), device, "ids")
    if scales is not None:
        _dense(scales, torch.float32, (n,), device, "scales")
    return K, n, r, N


def _bf16_matrix(t, T, C, device, name):
    """Row stride of a bf16 matrix [T, C]."""
    code, ld, own = _matrix(t, name)
    if code != _lib.OUT_BF16 or t.shape != (T, C) or own != device:
        raise ValueError(f"{name} must be a bf16 [{T}, {C}] tensor on device {device}, got {t.dtype} {list(t.shape)}")
    return ld


def lora_forward(x, down, up, ids, scales=None, base=None, out=None):
    """x bf16 [T, K], panels down bf16 [n, r, K] and up bf16 [n, r, N], ids int32 [T]
    -> (out bf16 [T, N], v): out[t] = base[t] + scales[a] up[a]^T (down[a] x[t]) with a
    = ids[t], and base[t] where ids[t] is outside [0, n).  scales: float32 [n], 1
    without; base: bf16 [T, N], 0 without; out may be base itself.  v: float32
    [splits, T, r rounded up to 4], the inner products in partial sums, which
    lora_backward takes."""
    device = _matrix(x, "x")[2]
    T = x.shape[0]
    K, n, r, N = _panels(down, up, T, ids, scales, device)
    ld = _bf16_matrix(x, T, K, device, "x")
    ld_base = 0 if base is None else _bf16_matrix(base, T, N, device, "base")
    if out is None:
        out, ld_out = x.new_empty((T, N)), N
    else:
        ld_out = _bf16_matrix(out, T, N, device, "out")
    v = x.new_empty((max(_lib.load().fp8mm_lora_splits(T, K, n, r), 1), T, (r + 3) // 4 * 4), dtype=torch.float32)
    _call("fp8mm_lora", x, x.data_ptr(), ld, T, K, down.data_ptr(), up.data_ptr(), n, r, N, ids.data_ptr(),
          _ptr(scales), _ptr(base), ld_base, out.data_ptr(), ld_out, v.data_ptr())
    return out, v


def lora_backward(dy, x, v, down, up, ids, scales=None, need_dx=True, need_down=True, need_up=True, out_dtype=None):
    """(dx, ddown, dup) of lora_forward from its x, v and panels; None where not
    needed.  dx: bf16 [T, K] (base's gradient is dy itself); ddown [n, r, K] and dup
    [n, r, N] have the panels' type, or out_dtype (bf16 or float32).  x may be None
    without need_down, v without need_up."""
    device = _matrix(dy, "dy")[2]
    T = dy.shape[0]
    K, n, r, N = _panels(down, up, T, ids, scales, device)
    ld_dy = _bf16_matrix(dy, T, N, device, "dy")
    lib = _lib.load()
    ld = 0
    if x is not None:
        ld = _bf16_matrix(x, T, K, device, "x")
    elif need_down:
        raise ValueError("x is needed for the gradient of down")
    if v is not None:
        splits = max(lib.fp8mm_lora_splits(T, K, n, r), 1)
        _dense(v, torch.float32, (splits, T, (r + 3) // 4 * 4), device, "v")
    elif need_up:
        raise ValueError("v is needed for the gradient of up")
    out_dtype = down.dtype if out_dtype is None else out_dtype
    code = _out_code(out_dtype)
    dx = dy.new_empty((T, K)) if need_dx else None
    ddown = dy.new_empty((n, r, K), dtype=out_dtype) if need_down else None
    dup = dy.new_empty((n, r, N), dtype=out_dtype) if need_up else None
    size = max(lib.fp8mm_lora_backward_workspace(T, K, N, n, r), 0)
    workspace = dy.new_empty((size,), dtype=torch.uint8)
    _call("fp8mm_lora_backward", dy, dy.data_ptr(), ld_dy, _ptr(x), ld, T, K, down.data_ptr(), up.data_ptr(), n, r, N,
          ids.data_ptr(), _ptr(scales), _ptr(v), _ptr(dx), K, _ptr(ddown), _ptr(dup), code, workspace.data_ptr(), size)
    return dx, ddown, dup


class _Lora(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, down, up, ids, scales, base):
        if ctx.needs_input_grad[4]:
            raise NotImplementedError("there is no gradient of the adapters' scales: pass scales.detach()")
        x, down, up, ids = x.contiguous(), down.contiguous(), up.contiguous(), ids.contiguous()
        scales = None if scales is None else scales.contiguous()
        base = None if base is None else base.contiguous()
        out, v = lora_forward(x, down, up, ids, scales, base)
        need = ctx.needs_input_grad
        ctx.save_for_backward(x if need[1] else None, v if need[2] else None, down, up, ids, scales)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, v, down, up, ids, scales = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = dy.to(torch.bfloat16).contiguous()
        grads = (None, None, None)
        if any(need[:3]):
            grads = lora_backward(g, x, v, down, up, ids, scales, *need[:3])
        return (*grads, None, None, g if need[5] else None)


def lora(x, down, up, ids, scales=None, base=None):
    """lora_forward's result, differentiable in x, down, up and base.  scales has no
    gradient: one that needs it is refused (NotImplementedError)."""
    if _differentiates(x, down, up, scales, base):
        return _Lora.apply(x, down, up, ids, scales, base)
    return lora_forward(x.contiguous(), down.contiguous(), up.contiguous(), ids.contiguous(),
                        None if scales is None else scales.contiguous(), None if base is None else base.contiguous())[0]
