"""Training operators: layer norm, the cross entropy of a linear head, AdamW.

What stands around a tropical product and its gradient (``gemm``,
``gemm_backward``, ``TropicalGemm``) when a model is trained with them.  Like
the rest of the package these functions marshal torch CUDA tensors into the C
ABI of ``include/tropical.h``; all computation runs in the library's kernels,
on the current stream or the one given (``stream``; copies and results too, as
under ``torch.cuda.stream``: the caller orders the inputs before the call and
the results' use after it).
"""

from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

import einsum_device_side_gb300 as _pkg

_CODES = {torch.float32: 0, torch.int32: 1, torch.int64: 2, torch.float64: 3, torch.bfloat16: 4, torch.float16: 5}
BLOCK = 256  # elements that share one scale of an 8-bit AdamW state


def _lib():
    return _pkg._lib or _pkg.load()


def _fast():
    """The CPython binding (the library loaded), or None where ctypes serves every call."""
    if _pkg._fc is None:
        _lib()
    return _pkg._fc


_empty, _empty_like, _f32 = torch.empty, torch.empty_like, torch.float32


def _fail(code: int, message: str):
    raise _pkg.TropicalError(code, message)


def _desc(t):
    """The C descriptor of a tensor, or None."""
    if t is None:
        return None
    d = _pkg.TropTensor()
    d.data = t.data_ptr() if t.numel() else None
    d.dtype = _CODES.get(t.dtype, -1)
    d.rank = t.dim()
    if d.rank:
        d.shape[:d.rank] = t.shape
        d.stride[:d.rank] = t.stride()
    return ctypes.byref(d)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _tensors(*values):
    for v in values:
        if isinstance(v, torch.Tensor):
            yield v
        elif isinstance(v, (list, tuple)):
            yield from _tensors(*v)


_OOM = -9


def _call(f, *args):
    """A call of the library.  Its workspace is not torch's: where there is no room for it, torch's allocator gives back
    what it keeps idle, and the call is made once more."""
    rc = f(*args)
    if rc == _OOM and not torch.cuda.is_current_stream_capturing():
        torch.cuda.empty_cache()
        rc = f(*args)
    return rc


def _stream_object(stream):
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream)


def _capturing(stream) -> bool:
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(_stream_object(stream)):
        return torch.cuda.is_current_stream_capturing()


def _on_stream(f, stream, *args, **kwargs):
    """``f`` with `stream` current: the copies it makes and the results it allocates then belong to the stream its kernels
    run on, in order with them.  The allocator is told of the tensors that one stream owns and the other uses, so that it
    hands out none of their memory while the other stream is not through with it."""
    stream = _stream_object(stream)
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        result = f(*args, **kwargs)
    if caller.cuda_stream != stream.cuda_stream:
        for t in _tensors(args, tuple(kwargs.values())):
            t.record_stream(stream)
        for t in _tensors(result):
            t.record_stream(caller)
    return result


def _check_vector(t, name: str, like, dtype, n: int):
    """A contiguous vector of n elements beside `like`, or None."""
    if t is None:
        return
    if t.dtype != dtype:
        _fail(-4, f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,):
        _fail(-5, f"{name} has shape {tuple(t.shape)}, not ({n},)")
    if t.get_device() != like.get_device():
        _fail(-3, f"{name} is on {t.device}, the operands on {like.device}")
    if not t.is_contiguous():
        _fail(-1, f"{name} must be contiguous")


def _result(x, dtype=None):
    """An uninitialised result of x's shape whose leading axes merge, whatever x's strides are."""
    return _empty_like(x, dtype=dtype or x.dtype) if x.dim() <= 2 else _empty(x.shape, dtype=dtype or x.dtype, device=x.device)


def _result_rows(t, n: int, c: int, name: str):
    """[..., C] as the matrix that a call writes."""
    try:
        return t.view(n, c)
    except RuntimeError:
        _fail(-10, f"{name}: the leading axes (shape {tuple(t.shape)}, strides {t.stride()}) must merge into one stride")


def _rows(t, name: str):
    """[..., C] as a matrix (a copy only where the leading axes do not merge into one stride)."""
    if t.dim() == 2:
        return t
    if t.dim() == 0:
        _fail(-1, f"{name} has no axis")
    return t.reshape(-1, t.shape[-1]) if t.numel() else t.new_empty((t.shape[:-1].numel(), t.shape[-1]))


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5, out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None, stream=None):
    """Layer norm over the last axis: ``(x - mean) * rstd * weight + bias``.

    ``x``: float32, bfloat16 or float16, its last axis contiguous, its leading axes in any order (where they do not merge
    into one stride, the rows are copied first; ``out``'s have to merge).  ``weight`` and ``bias`` are optional, of one type:
    x's or float32.  The result has x's type; a float32 ``x`` (a tropical product, say) may give ``out_dtype``
    bfloat16 or float16.  Returns ``(y, mean, rstd)``, the float32 statistics with x's leading shape:
    what ``layer_norm_backward`` reads."""
    if stream is not None:
        return _on_stream(layer_norm, stream, x, weight, bias, eps, out_dtype, out)
    fc = _fast()
    if out is None and out_dtype is None and fc is not None:  # the usual call
        r = fc.layer_norm(x, weight, bias, eps, stream)
        if r.__class__ is tuple:
            return r
        if r < 0:
            _pkg._check(r)
    if out is None:
        out = _result(x, out_dtype)
    elif out.shape != x.shape or (out_dtype is not None and out.dtype != out_dtype):
        _fail(-5, f"out is {tuple(out.shape)} {out.dtype}, not {tuple(x.shape)} {out_dtype or x.dtype}")
    mean = _empty(x.shape[:-1], dtype=_f32, device=x.device)
    rstd = _empty_like(mean)
    if fc is not None:
        rc = fc.layer_norm_t(x, weight, bias, eps, out, mean, rstd, stream)
        if rc == 0:
            return out, mean, rstd
        if rc < 0:
            _pkg._check(rc)
    x2 = _rows(x, "x")
    n, c = x2.shape
    w = weight if weight is not None else bias
    wdtype = w.dtype if w is not None else x.dtype
    _check_vector(weight, "weight", x, wdtype, c)
    _check_vector(bias, "bias", x, wdtype, c)
    _pkg._check(_lib().tropical_layer_norm(_desc(x2), _ptr(weight), _ptr(bias), _CODES.get(wdtype, -1), eps,
                                        _desc(_result_rows(out, n, c, "out")), _ptr(mean), _ptr(rstd), _pkg._stream(stream, x)))
    return out, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, *, want_x: bool = True, want_weight: bool = True,
                        want_bias: bool = True, weight_dtype: torch.dtype | None = None, stream=None):
    """Gradient of ``layer_norm``: ``(dx, dweight, dbias)``, an unwanted one None.  ``dy`` has the forward's result type;
    the weight's and bias's gradients have ``weight``'s type (``weight_dtype`` without one, by default x's)."""
    if stream is not None:
        return _on_stream(layer_norm_backward, stream, dy, x, mean, rstd, weight, want_x=want_x, want_weight=want_weight,
                          want_bias=want_bias, weight_dtype=weight_dtype)
    fc = _fast()
    if want_x and want_weight and want_bias and fc is not None and weight is not None:  # the usual call
        r = _call(fc.layer_norm_backward, dy, x, mean, rstd, weight, stream)
        if r.__class__ is tuple:
            return r
        if r < 0:
            _pkg._check(r)
    if dy.shape != x.shape:
        _fail(-5, f"dy has shape {tuple(dy.shape)}, x {tuple(x.shape)}")
    wdtype = weight.dtype if weight is not None else weight_dtype or x.dtype
    c = x.shape[-1]
    dx = _result(x) if want_x else None
    dw = _empty(c, dtype=wdtype, device=x.device) if want_weight else None
    db = None if not want_bias else _empty_like(dw) if want_weight else _empty(c, dtype=wdtype, device=x.device)
    if fc is not None:
        rc = _call(fc.layer_norm_backward_t, dy, x, mean, rstd, weight, dx, dw, db, stream)
        if rc == 0:
            return dx, dw, db
        if rc < 0:
            _pkg._check(rc)
    x2, dy2 = _rows(x, "x"), _rows(dy, "dy")
    n = x2.shape[0]
    _check_vector(weight, "weight", x, wdtype, c)
    _check_vector(mean.reshape(-1), "mean", x, torch.float32, n)
    _check_vector(rstd.reshape(-1), "rstd", x, torch.float32, n)
    if dy.get_device() != x.get_device():
        _fail(-3, f"dy is on {dy.device}, x on {x.device}")
    mean, rstd = mean.contiguous(), rstd.contiguous()
    _pkg._check(_call(_lib().tropical_layer_norm_backward, _desc(dy2), _desc(x2), _ptr(mean), _ptr(rstd), _ptr(weight),
                                                 _CODES.get(wdtype, -1), _desc(None if dx is None else dx.view(n, c)),
                                                 _ptr(dw), _ptr(db), _pkg._stream(stream, x)))
    return dx, dw, db


class LayerNorm(torch.autograd.Function):
    """Autograd over layer norm: ``LayerNorm.apply(x, weight, bias, eps, out_dtype)``.  First derivatives only: a second
    one (``create_graph=True``) raises."""

    @staticmethod
    def forward(ctx, x, weight=None, bias=None, eps=1e-5, out_dtype=None):
        y, mean, rstd = layer_norm(x, weight, bias, eps, out_dtype)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = (*ctx.needs_input_grad, False, False)  # (weight and bias may not have been given)
        dx, dw, db = layer_norm_backward(dy if dy.stride(-1) == 1 else dy.contiguous(), x, mean, rstd, weight,
                                         want_x=need[0], want_weight=need[1], want_bias=need[2],
                                         weight_dtype=ctx.bias_dtype)
        return dx, dw, db, None, None


_REDUCTIONS = {"none": 0, "mean": 1, "sum": 2}


def _check_head(x, w, target):
    if x.get_device() != w.get_device() or x.get_device() != target.get_device():
        _fail(-3, f"x is on {x.device}, w on {w.device}, target on {target.device}")


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, reduction: str = "mean",
                         ignore_index: int = -100, stream=None):
    """Softmax cross entropy of the logits ``x @ w.T`` without forming them in memory.

    ``x`` [N, D] and ``w`` [V, D]: both bfloat16 or both float16, any strides; ``target`` [N]: int32 or int64.  Returns
    ``(loss, lse, kept)``: the loss (one per token for ``reduction="none"``, else a scalar; tokens whose target is
    ``ignore_index`` have none), the log-sum-exp of each token's logits, and the number of tokens kept, all float32.
    A target outside the vocabulary gives NaN."""
    if stream is not None:
        return _on_stream(linear_cross_entropy, stream, x, w, target, reduction, ignore_index)
    fc = _fast()
    code = _REDUCTIONS.get(reduction)
    if code is None:
        _fail(-1, f"reduction must be one of {tuple(_REDUCTIONS)}, got {reduction!r}")
    if fc is not None:  # the usual call
        r = _call(fc.linear_ce, x, w, target, ignore_index, code, stream)
        if r.__class__ is tuple:
            return r
        if r < 0:
            _pkg._check(r)
    n = x.shape[0] if x.dim() else 0
    # (each a tensor of its own: a view could not be changed in place as an autograd function's result)
    total, kept = _empty((), dtype=_f32, device=x.device), _empty((), dtype=_f32, device=x.device)
    lse = _empty(n, dtype=_f32, device=x.device)
    loss = _empty_like(lse) if reduction == "none" else None
    each, mean = loss is not None, reduction == "mean"
    if fc is not None:
        rc = _call(fc.linear_ce_t, x, w, target, ignore_index, mean, loss, lse, None if each else total, kept, stream)
        if rc == 0:
            return loss if each else total, lse, kept
        if rc < 0:
            _pkg._check(rc)
    _check_head(x, w, target)
    _pkg._check(_call(_lib().tropical_linear_cross_entropy, _desc(x), _desc(w), _desc(target), ignore_index, mean, _ptr(loss),
                                                  _ptr(lse), None if each else _ptr(total), _ptr(kept),
                                                  _pkg._stream(stream, x)))
    return loss if each else total, lse, kept


def linear_cross_entropy_backward(dloss: torch.Tensor, x: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                                  lse: torch.Tensor, kept: torch.Tensor | None = None, ignore_index: int = -100, *,
                                  want_x: bool = True, want_w: bool = True, stream=None):
    """Gradient of ``linear_cross_entropy``: ``(dx, dw)`` in the operands' type, an unwanted one None.

    ``dloss``: float32, one per token or a scalar for all of them.  With ``kept`` (the mean's gradient) it is divided by
    that count.  The logits are formed again in pieces of the vocabulary; the workspace (512 MiB for a piece, besides sums
    and packed copies) stays the library's for the next call, until ``release_pool``."""
    if stream is not None:
        return _on_stream(linear_cross_entropy_backward, stream, dloss, x, w, target, lse, kept, ignore_index, want_x=want_x,
                          want_w=want_w)
    fc = _fast()
    dx = _empty(x.shape, dtype=x.dtype, device=x.device) if want_x else None
    dw = _empty(w.shape, dtype=w.dtype, device=w.device) if want_w else None
    if fc is not None:
        rc = _call(fc.linear_ce_backward_t, x, w, target, ignore_index, dloss, lse, kept, dx, dw, stream)
        if rc == 0:
            return dx, dw
        if rc < 0:
            _pkg._check(rc)
    _check_head(x, w, target)
    if dloss.dtype != torch.float32:
        _fail(-4, f"dloss must be float32, got {dloss.dtype}")
    if dloss.dim() > 1 or (dloss.dim() == 1 and dloss.shape[0] != x.shape[0]):
        _fail(-5, f"dloss has shape {tuple(dloss.shape)}: one per token or a scalar is wanted")
    _check_vector(lse, "lse", x, torch.float32, x.shape[0])
    if kept is not None and (kept.dtype != torch.float32 or kept.numel() != 1):
        _fail(-4, "kept must be one float32")
    for t, name in ((dloss, "dloss"), (kept, "kept")):
        if t is not None and t.get_device() != x.get_device():
            _fail(-3, f"{name} is on {t.device}, x on {x.device}")
    _pkg._check(_call(
        _lib().tropical_linear_cross_entropy_backward, _ptr(dloss), dloss.stride(0) if dloss.dim() else 0, _desc(x),
        _desc(w), _desc(target), ignore_index, _ptr(lse), _ptr(kept), _desc(dx), _desc(dw), _pkg._stream(stream, x)))
    return dx, dw


class LinearCrossEntropy(torch.autograd.Function):
    """Autograd over the head's loss: ``LinearCrossEntropy.apply(x, w, target, reduction, ignore_index)``.  First derivatives
    only: a second one (``create_graph=True``) raises."""

    @staticmethod
    def forward(ctx, x, w, target, reduction="mean", ignore_index=-100):
        loss, lse, kept = linear_cross_entropy(x, w, target, reduction, ignore_index)
        ctx.save_for_backward(x, w, target, lse, kept)
        ctx.reduction, ctx.ignore_index = reduction, ignore_index
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x, w, target, lse, kept = ctx.saved_tensors
        dx, dw = linear_cross_entropy_backward(dloss, x, w, target, lse, kept if ctx.reduction == "mean" else None,
                                               ctx.ignore_index, want_x=ctx.needs_input_grad[0],
                                               want_w=ctx.needs_input_grad[1])
        return dx, dw, None, None, None


class _Tensor(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                               "exp_avg_sq_scale", "copy")] + [("numel", ctypes.c_int64)]


class _State(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale",
                                               "exp_avg_value", "exp_avg_sq_value")] + [("numel", ctypes.c_int64)]


class _Options(ctypes.Structure):
    _fields_ = [(k, ctypes.c_double) for k in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + \
               [("step", ctypes.c_int64)]


def _column(ts, name: str, n: int, dtype, sizes, device):
    """The addresses of a list of contiguous tensors of one type and of these sizes."""
    if len(ts) != n:
        _fail(-5, f"{len(ts)} tensors in {name} for {n} parameters")
    out = []
    for i, (t, size) in enumerate(zip(ts, sizes)):
        if t.dtype != dtype:
            _fail(-4, f"{name}[{i}] must be {dtype}, got {t.dtype}")
        if t.numel() != size:
            _fail(-5, f"{name}[{i}] has {t.numel()} elements, not {size}")
        if t.get_device() != device:
            _fail(-3, f"{name}[{i}] is on {t.device}, the parameters on cuda:{device}")
        if not t.is_contiguous():
            _fail(-1, f"{name}[{i}] must be contiguous")
        out.append(t.data_ptr() or None)
    return out


def _table(params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies):
    n = len(params)
    if n == 0:
        return (_Tensor * 1)(), 0, 0, 0, 32, 0, [], -1
    sizes = [p.numel() for p in params]
    device, pdtype, gdtype = params[0].get_device(), params[0].dtype, grads[0].dtype if len(grads) else params[0].dtype
    if (exp_avg_scale is None) != (exp_avg_sq_scale is None):
        _fail(-1, "8-bit states have scales of both moments")
    bits = 32 if exp_avg_scale is None else 8
    mdtype, vdtype = (torch.float32, torch.float32) if bits == 32 else (torch.int8, torch.uint8)
    columns = {"param": _column(params, "params", n, pdtype, sizes, device),
               "grad": _column(grads, "grads", n, gdtype, sizes, device),
               "exp_avg": _column(exp_avg, "exp_avg", n, mdtype, sizes, device),
               "exp_avg_sq": _column(exp_avg_sq, "exp_avg_sq", n, vdtype, sizes, device)}
    if bits == 8:
        blocks = [-(-s // BLOCK) for s in sizes]
        columns["exp_avg_scale"] = _column(exp_avg_scale, "exp_avg_scale", n, torch.float32, blocks, device)
        columns["exp_avg_sq_scale"] = _column(exp_avg_sq_scale, "exp_avg_sq_scale", n, torch.float32, blocks, device)
    cdtype = 0
    if copies is not None and len(copies):
        cdtype = _CODES.get(copies[0].dtype, -1)
        columns["copy"] = _column(copies, "copies", n, copies[0].dtype, sizes, device)
    table = (_Tensor * n)()
    for i, e in enumerate(table):
        for k, v in columns.items():
            setattr(e, k, v[i])
        e.numel = sizes[i]
    return table, n, _CODES.get(pdtype, -1), _CODES.get(gdtype, -1), bits, cdtype, sizes, device


def _state_table(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, out):
    n = len(exp_avg)
    sizes = [t.numel() for t in exp_avg]
    blocks = [-(-s // BLOCK) for s in sizes]
    device = exp_avg[0].get_device() if n else -1
    columns = {"exp_avg": _column(exp_avg, "exp_avg", n, torch.int8, sizes, device),
               "exp_avg_sq": _column(exp_avg_sq, "exp_avg_sq", n, torch.uint8, sizes, device),
               "exp_avg_scale": _column(exp_avg_scale, "exp_avg_scale", n, torch.float32, blocks, device),
               "exp_avg_sq_scale": _column(exp_avg_sq_scale, "exp_avg_sq_scale", n, torch.float32, blocks, device),
               "exp_avg_value": _column(out[0], "out[0]", n, torch.float32, sizes, device),
               "exp_avg_sq_value": _column(out[1], "out[1]", n, torch.float32, sizes, device)}
    table = (_State * max(1, n))()
    for i in range(n):
        for k, v in columns.items():
            setattr(table[i], k, v[i])
        table[i].numel = sizes[i]
    return table, n


def adamw_step(params, grads, exp_avg, exp_avg_sq, exp_avg_scale=None, exp_avg_sq_scale=None, *, step: int,
               lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.01, grad_scale: float = 1.0, copies=None, stream=None):
    """One AdamW step over lists of tensors, in place; ``step`` counts from 1.

    ``params``: float32, bfloat16 or float16, all of one type; ``grads`` of one type (any for float32 parameters, else
    the parameters' or float32).  States: float32 like the parameters, or 8-bit codes (int8 ``exp_avg``, uint8
    ``exp_avg_sq``) with their float32 scales, one for every 256 elements.  ``copies``: 16-bit copies of float32
    parameters that the step writes too.  Every tensor is contiguous.  A program that steps the same tensors again and
    again keeps an ``AdamWPlan`` (or ``AdamW``), which reads the lists once."""
    if stream is not None:
        return _on_stream(adamw_step, stream, params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, step=step,
                          lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay, grad_scale=grad_scale,
                          copies=copies)
    lib = _lib()
    table, n, p, g, bits, c, _, device = _table(params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies)
    o = _Options(lr, beta1, beta2, eps, weight_decay, grad_scale, step)
    _pkg._check(lib.tropical_adamw_step(n, table, p, g, bits, c, ctypes.byref(o),
                                        _pkg._stream(stream, params[0] if n else None) if n else None))


def adamw_state_values(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, out=None, stream=None):
    """8-bit AdamW states as the values they stand for: two lists of float32 tensors (``out``: the lists to fill)."""
    if stream is not None:
        return _on_stream(adamw_state_values, stream, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, out)
    lib = _lib()
    if out is None:
        out = tuple([torch.empty(t.shape, dtype=torch.float32, device=t.device) for t in ts] for ts in (exp_avg, exp_avg_sq))
    table, n = _state_table(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, out)
    _pkg._check(lib.tropical_adamw_state_values(n, table, _pkg._stream(stream, exp_avg[0]) if n else None))
    return out


class AdamWPlan:
    """AdamW steps over the tensors given here (the lists of ``adamw_step``), checked and laid out once.  Like a tree plan
    it binds the buffers: ``step`` reads the gradients' current contents and updates parameters and states in place.
    ``values``: a pair of lists of float32 tensors that ``state_values`` fills from 8-bit states.  The tensors are kept
    referenced for the plan's lifetime."""

    def __init__(self, params, grads, exp_avg, exp_avg_sq, exp_avg_scale=None, exp_avg_sq_scale=None, *, copies=None,
                 values=None):
        lib = _lib()
        self._h = None
        lists = (params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies)
        table, n, p, g, bits, c, _, _ = _table(*lists)
        states = None
        if values is not None:
            if bits != 8:
                _fail(-1, "values of states that are not in 8 bits")
            states, _ = _state_table(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, values)
        h = ctypes.c_void_p()
        _pkg._check(_call(lib.tropical_adamw_plan_create, n, table, p, g, bits, c, states, ctypes.byref(h)))
        self._h = h.value
        self._keep = [None if t is None else list(t) for t in lists]
        self._streams = {}  # given to step or state_values: they use the tensors
        self._like = params[0] if n else torch.empty(0, device="cuda")
        self.values = values

    def step(self, step: int, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             weight_decay: float = 0.01, grad_scale: float = 1.0, stream=None):
        """One step; ``step`` counts from 1.  Captured into a CUDA graph it replays with this step number and these
        options: of use where the bias corrections are near 1."""
        if self._h is None:
            raise RuntimeError("plan is closed")
        if stream is not None:
            self._streams[stream.cuda_stream] = stream
        if _pkg._fc is not None:
            rc = _pkg._fc.adamw_plan_step(self._h, lr, beta1, beta2, eps, weight_decay, grad_scale, step, self._like,
                                          stream)
        else:
            o = _Options(lr, beta1, beta2, eps, weight_decay, grad_scale, step)
            rc = _pkg._lib.tropical_adamw_plan_step(self._h, ctypes.byref(o), _pkg._stream(stream, self._like))
        if rc:
            _pkg._check(rc)

    def state_values(self, stream=None):
        """Fills and returns ``values``."""
        if self._h is None:
            raise RuntimeError("plan is closed")
        if stream is not None:
            self._streams[stream.cuda_stream] = stream
        if _pkg._fc is not None:
            rc = _pkg._fc.adamw_plan_values(self._h, self._like, stream)
        else:
            rc = _pkg._lib.tropical_adamw_plan_values(self._h, _pkg._stream(stream, self._like))
        if rc:
            _pkg._check(rc)
        return self.values

    def close(self):
        if getattr(self, "_h", None) is not None:
            _pkg._check(_pkg._lib.tropical_adamw_plan_destroy(self._h))
            self._h = None
            for s in self._streams.values():  # steps that are still on their way: the memory is not handed out before
                for t in _tensors(self._keep, self.values):
                    t.record_stream(_stream_object(s))
            self._streams = {}

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AdamW:
    """AdamW with its states: ``AdamW(params, grads, state_bits=8)``, then ``step()`` whenever the gradients' buffers hold
    new ones.  ``grads`` are the buffers the backward pass writes (``p.grad`` of each parameter by default, which must
    exist and stay in place, ``zero_grad(set_to_none=False)``: a step finds out if it did not).  ``copies`` as in
    ``adamw_step``.  It counts its steps on the host, so a step cannot be captured into a CUDA graph (``AdamWPlan.step``
    can, with the step number given)."""

    def __init__(self, params, grads=None, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
                 eps: float = 1e-8, weight_decay: float = 0.01, state_bits: int = 32, copies=None):
        params = list(params)
        self._owners = params if grads is None else []
        if grads is None:
            grads = [p.grad for p in params]
            if any(g is None for g in grads):
                _fail(-1, "a parameter has no gradient buffer")
        params = [p.detach() for p in params]
        if state_bits not in (8, 32):
            _fail(-1, f"states of {state_bits} bits")
        new = lambda p, dtype, n=None: torch.zeros(p.shape if n is None else n, dtype=dtype, device=p.device)  # noqa: E731
        self.params, self.grads, self.steps = params, list(grads), 0
        self.options = dict(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        if state_bits == 32:
            self.exp_avg = [new(p, torch.float32) for p in params]
            self.exp_avg_sq = [new(p, torch.float32) for p in params]
        else:
            self.exp_avg = [new(p, torch.int8) for p in params]
            self.exp_avg_sq = [new(p, torch.uint8) for p in params]
            self.exp_avg_scale = [new(p, torch.float32, -(-p.numel() // BLOCK)) for p in params]
            self.exp_avg_sq_scale = [new(p, torch.float32, -(-p.numel() // BLOCK)) for p in params]
        self._plan = AdamWPlan(params, self.grads, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale,
                               self.exp_avg_sq_scale, copies=copies)

    def step(self, grad_scale: float = 1.0, stream=None):
        if _capturing(stream):
            _fail(-10, "a captured step would repeat its bias corrections at every replay: AdamW counts steps on the host")
        for i, (p, g) in enumerate(zip(self._owners, self.grads)):
            if p.grad is not g and (p.grad is None or p.grad.data_ptr() != g.data_ptr()):
                _fail(-1, f"parameter {i} has another gradient buffer than at first: clear gradients in place")
        self._plan.step(self.steps + 1, grad_scale=grad_scale, stream=stream, **self.options)
        self.steps += 1  # (a refused step does not count)
