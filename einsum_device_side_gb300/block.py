"""Operators of a residual block in training: its fused norms, activations kept in 8 bits.

They stand around a block of a deep network (a tropical product, say) as the
operators of ``train.py`` do around a single layer, and marshal torch CUDA
tensors into the C ABI of ``include/tropical.h`` in the same way: on the current
stream or the one given (``stream``; copies and results too).  ``Linear8`` alone
calls torch besides, for a plain linear layer's forward product and input gradient.
"""

from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

import einsum_device_side_gb300 as _pkg

from .train import _CODES, _call, _check_vector, _desc, _fail, _fast, _lib, _on_stream, _ptr, _result, _result_rows, _rows

GROUP = 32  # elements of a row that share one scale of an 8-bit copy


_empty, _empty_like, _f32, _i8, _u8 = torch.empty, torch.empty_like, torch.float32, torch.int8, torch.uint8


def _new_codes(shape, device):
    """Uninitialised codes and scales of a [..., C] activation.  Rows of codes start on 32 bytes: whole vectors for every
    kernel that reads them, whatever C is."""
    *lead, c = shape
    groups = -(-c // GROUP)
    codes = _empty((*lead, groups * GROUP), dtype=_i8, device=device)
    return codes if c == groups * GROUP else codes[..., :c], _empty((*lead, groups), dtype=_u8, device=device)


def _kept_rows(codes, scales, name: str):
    """Codes and scales [..., C] as matrices (copies only where the leading axes do not merge into one stride)."""
    if codes.dim() == 0 or scales.dim() == 0:
        _fail(-1, f"{name} has no axis")
    if codes.shape[:-1] != scales.shape[:-1]:
        _fail(-5, f"{name} has shape {tuple(codes.shape)}, its scales {tuple(scales.shape)}")
    if codes.get_device() != scales.get_device():
        _fail(-3, f"{name} is on {codes.device}, its scales on {scales.device}")
    return _rows(codes, name), _rows(scales, name)


def activation_pack(x: torch.Tensor, stream=None):
    """An activation in 8 bits, for the backward pass: ``(codes, scales)`` of ``x`` [..., C] (float32, bfloat16 or
    float16, last axis contiguous).

    Groups of 32 elements of a row share a power of two, ``unit = 2 ** (scale - 133)``, chosen so that the group's largest
    magnitude has 64 to 127 units; ``codes`` (int8, x's shape, rows on 32 bytes) are the elements over it, rounded to
    nearest, ``scales`` (uint8) [..., ceil(C / 32)].  An element is off by at most 1/128 of its group's largest magnitude.
    A group with an infinity or a NaN reads back as NaN."""
    if stream is not None:
        return _on_stream(activation_pack, stream, x)
    fc, codes, shape = _fast(), None, x.shape
    if fc is not None and len(shape) > 1:
        codes, scales = _new_codes(shape, x.device)
        if fc.activation_pack_t(x, codes, scales) == 0:  # the usual call
            return codes, scales
    lib = _lib()
    x2 = _rows(x, "x")
    if codes is None:
        codes, scales = _new_codes(x.shape, x.device)
    n, c = x2.shape
    _pkg._check(lib.tropical_activation_pack(_desc(x2), _desc(_result_rows(codes, n, c, "codes")),
                                             _desc(scales.view(n, -(-c // GROUP))), _pkg._stream(None, x)))
    return codes, scales


def activation_values(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None):
    """The values that an activation's 8-bit copy stands for, as ``dtype`` (bfloat16 and float32 hold them exactly; float16
    where they lie in its range)."""
    if stream is not None:
        return _on_stream(activation_values, stream, codes, scales, dtype)
    fc = _fast()
    out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    if fc is not None and codes.shape[:-1] == scales.shape[:-1] and fc.activation_values_t(codes, scales, out) == 0:  # the usual call
        return out
    lib = _lib()
    k2, s2 = _kept_rows(codes, scales, "codes")
    _pkg._check(lib.tropical_activation_values(_desc(k2), _desc(s2), _desc(out.view(k2.shape)), _pkg._stream(None, codes)))
    return out


def activation_weight_grad(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out_dtype: torch.dtype | None = None,
                           want_bias: bool = False, stream=None):
    """The weight gradient of a linear layer ``y = x @ w.T + b`` whose input was kept in 8 bits: ``(dw, db)``,
    ``dw = dy.T @ x`` [O, C] and, if wanted, ``db`` [O], the sum of ``dy``'s rows.

    ``dy`` [..., O]: bfloat16 or float16, any strides; ``codes``, ``scales``: ``activation_pack`` of x [..., C], whose
    values enter in dy's type (bfloat16 holds them exactly; float16 makes infinities of those outside its range).  Sums are
    float32; results have dy's type or float32 (``out_dtype``)."""
    if stream is not None:
        return _on_stream(activation_weight_grad, stream, dy, codes, scales, out_dtype, want_bias)
    fc = _fast()
    if fc is not None and dy.dim() == codes.dim() == scales.dim() == 2 and dy.shape[0] == codes.shape[0] == scales.shape[0]:  # the usual call
        dw = torch.empty((dy.shape[1], codes.shape[1]), dtype=out_dtype or dy.dtype, device=dy.device)
        db = torch.empty(dy.shape[1], dtype=dw.dtype, device=dy.device) if want_bias else None
        if fc.activation_weight_grad_t(dy, codes, scales, dw, db) == 0:
            return dw, db
    lib = _lib()
    k2, s2 = _kept_rows(codes, scales, "codes")
    if codes.shape[:-1] != dy.shape[:-1]:
        _fail(-5, f"dy has shape {tuple(dy.shape)}, codes {tuple(codes.shape)}")
    if dy.get_device() != codes.get_device():
        _fail(-3, f"dy is on {dy.device}, codes on {codes.device}")
    dy2 = _rows(dy, "dy")
    out_dtype = out_dtype or dy.dtype
    dw = torch.empty((dy2.shape[1], k2.shape[1]), dtype=out_dtype, device=dy.device)
    db = torch.empty(dy2.shape[1], dtype=out_dtype, device=dy.device) if want_bias else None
    _pkg._check(_call(lib.tropical_activation_weight_grad, _desc(dy2), _desc(k2), _desc(s2), _desc(dw), _ptr(db),
                      _pkg._stream(None, dy)))
    return dw, db


class Linear8(torch.autograd.Function):
    """A linear layer that keeps its input in 8 bits: ``Linear8.apply(x, w, bias)`` is ``x @ w.T + bias``, its weight's and
    bias's gradients come from the copy (``activation_weight_grad``).  The product itself and x's gradient are torch's matmul.  ``x`` [..., C], ``w`` [O, C] and ``bias`` [O] or
    None: all bfloat16 or all float16.  First derivatives only: a second one (``create_graph=True``) raises."""

    @staticmethod
    def forward(ctx, x, w, bias=None):
        if x.dtype not in (torch.bfloat16, torch.float16) or w.dtype != x.dtype or (bias is not None and bias.dtype != x.dtype):
            _fail(-4, f"x is {x.dtype}, w {w.dtype}, bias {None if bias is None else bias.dtype}: one 16-bit type is wanted")
        ctx.has_bias = bias is not None
        wanted = ctx.needs_input_grad[1] or (ctx.has_bias and ctx.needs_input_grad[2])
        codes = activation_pack(x if x.stride(-1) == 1 else x.contiguous()) if wanted else (None, None)
        ctx.save_for_backward(w, *codes)
        return torch.nn.functional.linear(x, w, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w, codes, scales = ctx.saved_tensors
        need = (*ctx.needs_input_grad, False)
        dx = dy @ w if need[0] else None
        dw = db = None
        if codes is not None:
            dw, db = activation_weight_grad(dy, codes, scales, want_bias=need[2])
        return (dx, dw if need[1] else None, db)[:len(ctx.needs_input_grad)]


_NONE_KEPT = (None,) * 6
_NORMS = {"layer": 0, "rms": 1}
_ACTS = {"none": 0, "sigmoid": 1, "silu": 2}


class _Options(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int) for k in ("norm", "post_norm", "gate_act", "wdtype")] + \
               [(k, ctypes.c_double) for k in ("alpha", "scale", "eps")] + \
               [(k, ctypes.c_void_p) for k in ("weight", "bias", "post_weight", "post_bias", "scale_vector")]


_TENSOR = ctypes.POINTER(_pkg.TropTensor)


class _Kept(ctypes.Structure):
    _fields_ = [("codes", _TENSOR), ("scales", _TENSOR)]


class _Grads(ctypes.Structure):
    _fields_ = [(k, _TENSOR) for k in ("dx", "du", "dgate")] + \
               [(k, ctypes.c_void_p) for k in ("dscale", "dweight", "dbias", "dpost_weight", "dpost_bias")]


def _pointer(t):
    d = _desc(t)
    return None if d is None else ctypes.pointer(d._obj)


def _options(weight, bias, post_weight, post_bias, scale, post_norm, norm, gate_act, alpha, eps):
    """The options' values in the order that the bindings take them; the vectors as they were given."""
    if norm not in _NORMS or gate_act not in _ACTS:
        _fail(-1, f"norm must be one of {tuple(_NORMS)}, gate_act one of {tuple(_ACTS)}, got {norm!r} and {gate_act!r}")
    vector = scale if isinstance(scale, torch.Tensor) else None
    return (_NORMS[norm], 1 if post_norm else 0, _ACTS[gate_act], alpha, 1.0 if scale is None or vector is not None else scale, eps,
            weight, bias, post_weight, post_bias, vector)


def _options_struct(values, like, c, wdtype):
    """The C options, their vectors checked."""
    for v, name in zip(values[6:], ("weight", "bias", "post_weight", "post_bias", "scale")):
        _check_vector(v, name, like, wdtype, c)
    return _Options(*values[:3], _CODES.get(wdtype, -1), *values[3:6], *map(_ptr, values[6:]))


def _vector_type(values, otherwise):
    return next((v.dtype for v in values[6:] if v is not None), otherwise)


def _beside(t, name: str, like, shape):
    """A tensor of this shape on the same device."""
    if t.shape != shape:
        _fail(-5, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.get_device() != like.get_device():
        _fail(-3, f"{name} is on {t.device}, the operands on {like.device}")


def _gate_rows(gate, like, shape):
    if gate is None:
        return None
    if gate.dim() != len(shape) or gate.shape[:-1] != shape[:-1] or gate.shape[-1] not in (1, shape[-1]):
        _fail(-5, f"gate has shape {tuple(gate.shape)}: {tuple(shape)}, or 1 in the last place, is wanted")
    if gate.get_device() != like.get_device():
        _fail(-3, f"gate is on {gate.device}, the operands on {like.device}")
    return _rows(gate, "gate")


def residual_norm(x: torch.Tensor, u: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                  gate: torch.Tensor | None = None, gate_act: str = "none", scale: float | torch.Tensor | None = None,
                  post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None, post_norm: bool = True,
                  norm: str = "layer", alpha: float = 1.0, eps: float = 1e-5, out_dtype: torch.dtype | None = None,
                  keep: bool = False, stream=None):
    """What lies between one block's output and the next block's input, in one pass over memory:

        v = norm(u) * post_weight + post_bias        (``post_norm=False``: v = u)
        r = alpha * x + scale * act(gate) * v
        y = norm(r) * weight + bias

    ``x`` [..., C]: the residual stream; ``u``: the block's output.  ``gate``: x's shape, or one value a row [..., 1];
    ``gate_act``: "none", "sigmoid" or "silu".  ``scale``: a number or a vector [C].  ``norm``: "layer" or "rms" (both
    norms).  Types float32, bfloat16 or float16: u's and gate's are x's, or 16-bit beside a float32 x; y's is u's, or
    ``out_dtype`` 16-bit beside a float32 u; the vectors are of y's type or float32.  Last axes are contiguous; leading
    axes lie in any order (rows that do not merge into one stride are copied first).

    Returns ``(y, r, stats, kept)``: the next block's input, the new stream (x's type), float32 statistics
    [4, ...leading] (mean and 1/deviation of u, then of r), which the backward pass reads, and with ``keep`` 8-bit copies of
    what it reads besides, ``(u, gate, r)`` for ``residual_norm_backward``: pairs as ``activation_pack`` returns them (of r
    as it is stored; a gate of one value a row and None stay what they are).  Without ``keep`` that is None."""
    if stream is not None:
        return _on_stream(residual_norm, stream, x, u, weight, bias, gate=gate, gate_act=gate_act, scale=scale,
                          post_weight=post_weight, post_bias=post_bias, post_norm=post_norm, norm=norm, alpha=alpha, eps=eps,
                          out_dtype=out_dtype, keep=keep)
    values = _options(weight, bias, post_weight, post_bias, scale, post_norm, norm, gate_act, alpha, eps)
    shape, device = x.shape, x.device
    if not shape:
        _fail(-1, "x has no axis")
    *lead, c = shape
    y, r = _result(u, out_dtype), _result(x)
    stats = _empty((4, *lead), dtype=_f32, device=device)
    kept, copies, full = None, _NONE_KEPT, False
    if keep:
        full = gate is not None and gate.dim() > 0 and gate.shape[-1] == c
        ku, kr = _new_codes(shape, device), _new_codes(shape, device)
        kg = _new_codes(shape, device) if full else gate
        kept, copies = (ku, kg, kr), (*ku, *(kg if full else (None, None)), *kr)
    fc = _fast()
    if fc is not None and fc.residual_norm_t(*values, x, u, gate, y, r, stats, *copies) == 0:  # the usual call
        return y, r, stats, kept
    lib = _lib()
    x2, u2 = _rows(x, "x"), _rows(u, "u")
    n = x2.shape[0]
    _beside(u, "u", x, shape)
    g2 = _gate_rows(gate, x, shape)
    o = _options_struct(values, x, c, _vector_type(values, x.dtype))
    table, _held = _kept_table(ku, kg if full else None, kr) if keep else (None, None)
    _pkg._check(lib.tropical_residual_norm(ctypes.byref(o), _desc(x2), _desc(u2), _desc(g2), _desc(_result_rows(y, n, c, "y")),
                                           _desc(_result_rows(r, n, c, "r")), _ptr(stats), table, _pkg._stream(None, x)))
    return y, r, stats, kept


def _kept_table(*pairs):
    """The C table of u's, the gate's and r's copies, and the matrices it points to (to be held until the call)."""
    table, held = (_Kept * 3)(), []
    for to, pair in zip(table, pairs):
        if pair is not None:
            held.append(_kept_rows(*pair, "an 8-bit copy"))
            to.codes, to.scales = map(_pointer, held[-1])
    return table, held


_GRADS = ("x", "u", "gate", "scale", "weight", "bias", "post_weight", "post_bias")
_ALL_GRADS = frozenset(_GRADS)


def residual_norm_backward(dy: torch.Tensor, dr: torch.Tensor | None, r, u, stats: torch.Tensor,
                           weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *, gate=None,
                           gate_act: str = "none", scale: float | torch.Tensor | None = None,
                           post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
                           post_norm: bool = True, norm: str = "layer", alpha: float = 1.0, want=None,
                           x_dtype: torch.dtype | None = None, u_dtype: torch.dtype | None = None, stream=None):
    """Gradient of ``residual_norm``: ``(dx, du, dgate, dscale, dweight, dbias, dpost_weight, dpost_bias)``, one for every
    tensor given (``bias`` is not read but for that) and None for the others; ``want``: the names of those to compute, of
    "x", "u", "gate", "scale", "weight", "bias", "post_weight", "post_bias".

    ``dy``: y's gradient; ``dr``: what reaches r from elsewhere, or None; ``stats``: the forward call's, [4, ...leading].  ``r``,
    ``u`` and ``gate``: as the forward call had them, or their 8-bit copies (pairs; a gate of one value a row stays as it is).  From copies the gradients' types are
    ``x_dtype`` (by default dr's, else dy's) and ``u_dtype`` (dy's)."""
    if stream is not None:
        return _on_stream(residual_norm_backward, stream, dy, dr, r, u, stats, weight, bias, gate=gate, gate_act=gate_act,
                          scale=scale, post_weight=post_weight, post_bias=post_bias, post_norm=post_norm, norm=norm,
                          alpha=alpha, want=want, x_dtype=x_dtype, u_dtype=u_dtype)
    values = _options(weight, bias, post_weight, post_bias, scale, post_norm, norm, gate_act, alpha, 0.0)
    if want is None:
        want = _ALL_GRADS
    elif not _ALL_GRADS.issuperset(want := {want} if isinstance(want, str) else set(want)):
        _fail(-1, f"want must name some of {_GRADS}, got {sorted(map(str, want - _ALL_GRADS))}")
    shape, device = dy.shape, dy.device
    if not shape:
        _fail(-1, "dy has no axis")
    *lead, c = shape
    if stats.shape != (4, *lead) and stats.shape != (4, math.prod(lead)):  # (as a matrix of the rows: the same in memory)
        _fail(-5, f"stats has shape {tuple(stats.shape)}, not {(4, *lead)}")
    copies, coded = isinstance(r, tuple), isinstance(gate, tuple)
    if copies != isinstance(u, tuple):
        _fail(-1, "r and u are both 8-bit copies, or neither is")
    if coded and not copies:
        _fail(-1, "the gate's 8-bit copy without r's and u's")
    if copies:
        x_dtype = x_dtype or (dr.dtype if dr is not None else dy.dtype)
        u_dtype = u_dtype or dy.dtype
    else:
        x_dtype, u_dtype = r.dtype, u.dtype
    wdtype = _vector_type(values, dy.dtype)
    new = lambda name, dtype, cols=c: _empty((*lead, cols), dtype=dtype, device=device) if name in want else None  # noqa: E731
    vec = lambda name, v: _empty_like(v) if v is not None and name in want else None  # noqa: E731
    dx, du = new("x", x_dtype), new("u", u_dtype)
    dgate = None if gate is None else new("gate", u_dtype, ((gate[0] if coded else gate).shape or (1,))[-1])
    vectors = [vec("scale", values[10]), vec("weight", weight), vec("bias", bias), vec("post_weight", post_weight),
               vec("post_bias", post_bias)]
    plain = None if coded else gate
    types = _CODES.get(x_dtype, -1), _CODES.get(u_dtype, -1)
    fc = _fast()
    if fc is not None:
        given = (None, None, plain) if copies else (r, u, plain)
        kept = (*u, *(gate if coded else (None, None)), *r) if copies else _NONE_KEPT
        if fc.residual_norm_backward_t(*values, dy, dr, *given, stats, *kept, dx, du, dgate, *vectors, *types) == 0:  # the usual call
            return dx, du, dgate, *vectors
    lib = _lib()
    dy2 = _rows(dy, "dy")
    n = dy2.shape[0]
    r2 = u2 = table = None
    if copies:
        for pair, name in ((r, "r"), (u, "u"), (gate if coded else r, "gate")):
            _beside(pair[0], name, dy, shape)
        table, _held = _kept_table(u, gate if coded else None, r)
    else:
        _beside(r, "r", dy, shape)
        _beside(u, "u", dy, shape)
        r2, u2 = _rows(r, "r"), _rows(u, "u")
    g2 = _gate_rows(plain, dy, shape)
    if dr is not None:
        _beside(dr, "dr", dy, shape)
    _check_vector(stats.reshape(-1), "stats", dy, torch.float32, 4 * n)
    o = _options_struct(values, dy, c, wdtype)
    dr2, stats = None if dr is None else _rows(dr, "dr"), stats.contiguous()
    flat = lambda t: None if t is None else _pointer(t.view(n, t.shape[-1]))  # noqa: E731
    grads = _Grads(flat(dx), flat(du), flat(dgate), *[_ptr(v) for v in vectors])
    _pkg._check(_call(lib.tropical_residual_norm_backward, ctypes.byref(o), _desc(dy2), _desc(dr2), _desc(r2), _desc(u2),
                      _desc(g2), _ptr(stats), table, *types, ctypes.byref(grads), _pkg._stream(None, dy)))
    return dx, du, dgate, *vectors


class ResidualNorm(torch.autograd.Function):
    """Autograd over ``residual_norm``: ``y, r = ResidualNorm.apply(x, u, weight, bias, gate, gate_act, scale, post_weight,
    post_bias, post_norm, norm, alpha, eps, out_dtype, keep)``, with the function's meanings and defaults.  With ``keep`` the
    8-bit copies are what it holds for the backward pass; else u, gate and r.  First derivatives only: a second one
    (``create_graph=True``) raises."""

    @staticmethod
    def forward(ctx, x, u, weight=None, bias=None, gate=None, gate_act="none", scale=None, post_weight=None, post_bias=None,
                post_norm=True, norm="layer", alpha=1.0, eps=1e-5, out_dtype=None, keep=False):
        y, r, stats, kept = residual_norm(x, u, weight, bias, gate=gate, gate_act=gate_act, scale=scale,
                                          post_weight=post_weight, post_bias=post_bias, post_norm=post_norm, norm=norm,
                                          alpha=alpha, eps=eps, out_dtype=out_dtype, keep=keep)
        held = (u, gate, r) if kept is None else kept
        ctx.pairs = [isinstance(t, tuple) for t in held]
        ctx.vector = isinstance(scale, torch.Tensor)
        flat = [t for pair in held for t in (pair if isinstance(pair, tuple) else (pair,))]
        ctx.save_for_backward(stats, weight, bias, post_weight, post_bias, scale if ctx.vector else None, *flat)
        ctx.scale = None if ctx.vector else scale
        ctx.options = dict(gate_act=gate_act, post_norm=post_norm, norm=norm, alpha=alpha, x_dtype=x.dtype, u_dtype=u.dtype)
        ctx.y_like = y.shape, y.dtype, y.device
        ctx.set_materialize_grads(False)
        return y, r

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr):
        stats, weight, bias, post_weight, post_bias, vector, *flat = ctx.saved_tensors
        flat = iter(flat)
        u, gate, r = [(next(flat), next(flat)) if pair else next(flat) for pair in ctx.pairs]
        if dy is None:
            shape, dtype, device = ctx.y_like
            dy = torch.zeros(shape, dtype=dtype, device=device)
        rows = lambda t: t if t is None or t.stride(-1) == 1 else t.contiguous()  # noqa: E731
        need = (*ctx.needs_input_grad, *[False] * 15)  # (later arguments may not have been given)
        want = {name for name, i in zip(_GRADS, (0, 1, 4, 6, 2, 3, 7, 8)) if need[i]}
        dx, du, dgate, dscale, dweight, dbias, dpw, dpb = residual_norm_backward(
            rows(dy), rows(dr), r, u, stats, weight, bias, gate=gate, scale=vector if ctx.vector else ctx.scale,
            post_weight=post_weight, post_bias=post_bias, want=want, **ctx.options)
        grads = (dx, du, dweight, dbias, dgate, None, dscale, dpw, dpb, None, None, None, None, None, None)
        return grads[:len(ctx.needs_input_grad)]
