"""Layer norm, root-mean-square norm and embedding: forward and backward calls
of the C ABI.

Like the rest of the binding these functions only marshal arguments.  Tensors
are float32, bfloat16 or float16 on one HIP device; every call runs on the
current stream of that device, allocates its outputs and scratch from torch's
allocator (so it can be captured in a HIP graph) and does not synchronise.
``layer_norm``, ``rms_norm`` and ``embedding`` take part in autograd: their
gradients are ``layer_norm_backward``, ``rms_norm_backward`` and
``embedding_backward``, which are plain calls without a derivative of their
own.  There is no forward-mode derivative: a dual tensor is refused
(``NotImplementedError``).

A captured backward pass is subject to torch's own rule: no eager graph of
the same leaves may be alive while it is captured, as their gradients would
then be ordered against the eager graph's stream, outside the capture.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator

import torch
from torch.autograd import forward_ad

from . import SvError, _check, capi, short_way as native

__all__ = ["layer_norm", "layer_norm_backward", "rms_norm", "rms_norm_fp8", "rms_norm_backward", "embedding",
           "embedding_backward"]

_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_TYPES = tuple(_CODES)
_UNSUPPORTED = ctypes.c_size_t(-1).value
_HERE = contextlib.nullcontext()
# the raw stream handle without a Stream object, where torch has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _tensor(t, name, dtypes):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")


def _no_tangents(*tensors):
    """Refuses dual tensors: no forward-mode derivative is computed here, and a
    result without its tangent would pass for a constant."""
    if forward_ad._current_level >= 0 and any(
            isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError("the norms and the embedding have no forward-mode derivative")


def _same_device(ref, t, name):
    if t.get_device() != ref.get_device():  # both on HIP devices, as _tensor has checked
        raise ValueError(f"{name} is on {t.device}, the other tensors on {ref.device}")


def _on(device):
    """The tensors' device, current for the launches and the allocations."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stored(t):
    """t's values, contiguous in memory.  Torch negates some views as it reads
    them (imaginary parts of conjugates): their memory holds the opposite."""
    return (t.detach().resolve_neg() if t.is_neg() else t).contiguous()


def _rows(t, rows, n):
    """t as [rows, n] with contiguous rows (a view where its strides allow
    one, else a copy), and its row stride."""
    if t.is_neg():
        t = _stored(t)
    if t.is_contiguous():
        return t, n
    t = t.detach().reshape(rows, n)
    if rows == 0 or n == 0:
        return t, n
    if (n > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < n):
        t = t.contiguous()
    return t, t.stride(0) if rows > 1 else n


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scratch(nbytes, device, what):
    if nbytes == _UNSUPPORTED:
        raise SvError(5, f"{what}: this shape is not supported")
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _shape_2d(x, name):
    if x.dim() < 1:
        raise ValueError(f"{name} needs at least one dimension")
    n = x.shape[-1]
    return math.prod(x.shape[:-1]), n


# ---------------------------------------------------------------- layer norm

def _param(t, name, x, n, dtype=None):
    _tensor(t, name, (x.dtype, torch.float32) if x.dtype != torch.float32 else (torch.float32,))
    _same_device(x, t, name)
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"weight and bias must have one type, got {dtype} and {t.dtype}")
    return _stored(t)


def _norm_forward(x, weight, bias, eps, stats):
    rows, n = _shape_2d(x, "x")
    w = _param(weight, "weight", x, n) if weight is not None else None
    b = _param(bias, "bias", x, n, w.dtype if w is not None else None) if bias is not None else None
    pt = w.dtype if w is not None else b.dtype if b is not None else torch.float32
    x2, ldx = _rows(x, rows, n)
    with _on(x.device):
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        mean = rstd = None
        if stats:
            mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
            rstd = torch.empty_like(mean)
        _check(capi().sv_layer_norm(_ptr(x2), _CODES[x.dtype], rows, n, ldx, _ptr(w), _ptr(b), _CODES[pt], eps,
                                    _ptr(y), n, _ptr(mean), _ptr(rstd),
                                    _raw_stream(x.device.index)))
    return y, mean, rstd


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _norm_forward(x, weight, bias, eps, True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = bias.dtype if bias is not None else None
        ctx.mark_non_differentiable(mean, rstd)
        return y, mean, rstd

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, _mean, _rstd):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b, _ = ctx.needs_input_grad
        dx, dw, db = _norm_backward(dy, x, mean, rstd, weight, need_x, need_w, need_b,
                                    weight.dtype if weight is not None else ctx.bias_dtype)
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, return_stats: bool = False):
    """Layer norm over the last dimension: ``(x - mean) / sqrt(var + eps) *
    weight + bias``, with the variance's shift, local centring and two-term
    correction, computed in float32 and rounded once to x's type.

    ``weight`` and ``bias`` (each optional) have shape ``[n]`` and one type,
    x's or float32.  With ``return_stats`` also the mean and
    ``1 / sqrt(var + eps)`` of each row (float32, not differentiable), which
    ``layer_norm_backward`` takes.  Rows may be strided; a last dimension that
    is not contiguous is copied first.  A row's result does not depend on the
    other rows.
    """
    _tensor(x, "x", _TYPES)
    _no_tangents(x, weight, bias)
    eps = float(eps)
    # what is no tensor is refused where the parameters are checked
    if torch.is_grad_enabled() and (x.requires_grad or getattr(weight, "requires_grad", False)
                                    or getattr(bias, "requires_grad", False)):
        y, mean, rstd = _LayerNorm.apply(x, weight, bias, eps)
    else:
        y, mean, rstd = _norm_forward(x, weight, bias, eps, return_stats)
    return (y, mean, rstd) if return_stats else y


def _norm_backward(dy, x, mean, rstd, weight, need_x, need_w, need_b, param_dtype):
    _no_tangents(dy, x, mean, rstd, weight)
    rows, n = _shape_2d(x, "x")
    w = _param(weight, "weight", x, n) if weight is not None else None
    dy2, lddy = _rows(dy, rows, n)
    x2, ldx = _rows(x, rows, n)
    mean, rstd = _stored(mean), _stored(rstd)
    L = capi()
    with _on(x.device):
        dx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_x else None
        dw = torch.empty(n, dtype=param_dtype, device=x.device) if need_w else None
        db = torch.empty(n, dtype=param_dtype, device=x.device) if need_b else None
        nbytes = L.sv_layer_norm_backward_workspace_size(rows, n, _CODES[x.dtype]) if need_w or need_b else 0
        ws = _scratch(nbytes, x.device, "layer_norm_backward")
        _check(L.sv_layer_norm_backward(_ptr(dy2), lddy, _ptr(x2), ldx, _CODES[x.dtype], rows, n, _ptr(w),
                                        _CODES[param_dtype if param_dtype is not None else torch.float32], _ptr(mean),
                                        _ptr(rstd), _ptr(dx), n, _ptr(dw), _ptr(db), _ptr(ws), nbytes,
                                        _raw_stream(x.device.index)))
    return dx, dw, db


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, weight_grad: bool = True, bias_grad: bool = True,
                        param_dtype=None):
    """Gradients ``(dx, dweight, dbias)`` of ``layer_norm`` at x for the
    gradient ``dy`` of its result, from the ``mean`` and ``rstd`` it returned.

    ``dweight`` and ``dbias`` have the weight's type (``param_dtype``, x's
    type or float32, when there is no weight; float32 by default) and are
    None where not asked for.
    """
    _tensor(x, "x", _TYPES)
    _tensor(dy, "dy", (x.dtype,))
    _same_device(x, dy, "dy")
    if dy.shape != x.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, x {tuple(x.shape)}")
    _shape_2d(x, "x")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _tensor(t, name, (torch.float32,))
        _same_device(x, t, name)
        if t.shape != x.shape[:-1]:
            raise ValueError(f"{name} must have shape {tuple(x.shape[:-1])}, got {tuple(t.shape)}")
    if weight is not None:
        _tensor(weight, "weight", (x.dtype, torch.float32))
        if param_dtype not in (None, weight.dtype):
            raise TypeError(f"param_dtype {param_dtype} differs from the weight's {weight.dtype}")
        param_dtype = weight.dtype
    elif param_dtype is None:
        param_dtype = torch.float32
    elif param_dtype not in (x.dtype, torch.float32):
        raise TypeError(f"param_dtype must be {x.dtype} or torch.float32, got {param_dtype}")
    return _norm_backward(dy, x, mean, rstd, weight, True, bool(weight_grad), bool(bias_grad), param_dtype)


# ---------------------------------------------------------------- root-mean-square norm

_FP8 = {torch.float8_e4m3fn: 3, torch.float8_e5m2: 4}
_BLOCK = 128  # values that share a scale


def _short(x, weight, eps, residual, want_rstd, out_code=0, block=0):
    """The call for ordinary tensors (rows in order in memory, on the current
    device, nothing to record), None for others."""
    if forward_ad._current_level >= 0:
        return None
    return native().rms(x, weight, residual, eps, want_rstd, out_code, block)


def _rms_inputs(x, weight, residual, rows, n):
    """Checked and stored: x, its row stride, the residual, its row stride and
    type code, the weight and its type."""
    w = _param(weight, "weight", x, n) if weight is not None else None
    x2, ldx = _rows(x, rows, n)
    if residual is None:
        return x2, ldx, None, n, _CODES[x.dtype], w
    _tensor(residual, "residual", (x.dtype, torch.float32) if x.dtype != torch.float32 else (torch.float32,))
    _same_device(x, residual, "residual")
    if residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")
    r2, ldr = _rows(residual, rows, n)
    return x2, ldx, r2, ldr, _CODES[residual.dtype], w


def _rms_forward(x, weight, eps, residual, want_rstd):
    rows, n = _shape_2d(x, "x")
    x2, ldx, r2, ldr, sum_code, w = _rms_inputs(x, weight, residual, rows, n)
    code = _CODES[x.dtype]
    with _on(x.device):
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        h = None if residual is None else torch.empty_like(residual, memory_format=torch.contiguous_format)
        rstd = x.new_empty(x.shape[:-1], dtype=torch.float32) if want_rstd else None
        _check(capi().sv_rms_norm(_ptr(x2), ldx, _ptr(r2), ldr, code, sum_code, rows, n, _ptr(w),
                                  code if w is None else _CODES[w.dtype], eps, _ptr(y), n, _ptr(h), n, _ptr(rstd),
                                  _raw_stream(x.device.index)))
    return y, h, rstd


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = _rms_forward(x, weight, eps, residual, True)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        ctx.x_dtype = x.dtype
        ctx.mark_non_differentiable(rstd)
        ctx.set_materialize_grads(False)
        return y, h, rstd

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dsum, _rstd):
        h, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r, _ = ctx.needs_input_grad
        mixed = h.dtype != ctx.x_dtype
        if dy is None:  # y took no part
            dx = dsum.to(ctx.x_dtype) if need_x and dsum is not None else None
            return dx, None, dsum if need_r else None, None
        args = dy, h, rstd, weight, dsum, need_r or (need_x and not mixed), need_x and mixed, need_w
        dh, dx, dw = _short_backward(*args) or _rms_backward(*args, weight.dtype if weight is not None else None)
        return dx if mixed else dh if need_x else None, dw, dh if need_r else None, None


def rms_norm(x, weight=None, eps: float = 1e-6, residual=None, return_rstd: bool = False):
    """Root-mean-square norm over the last dimension: ``x / sqrt(mean(x^2) +
    eps) * weight``, the squares summed in float64, the rest computed in
    float32 and rounded once to x's type.

    With a ``residual`` (x's shape; x's type or float32) the norm is of ``h =
    x + residual``, rounded to the residual's type, and ``(y, h)`` is returned.
    ``weight`` (optional) has shape ``[n]`` and x's type or float32.  With
    ``return_rstd`` also ``1 / sqrt(mean(h^2) + eps)`` of each row (float32,
    not differentiable), which ``rms_norm_backward`` takes.  Rows may be
    strided; a last dimension that is not contiguous is copied first.  A row's
    result does not depend on the other rows.
    """
    eps = float(eps)
    out = _short(x, weight, eps, residual, return_rstd)
    if out is not None:
        return out
    _tensor(x, "x", _TYPES)
    _no_tangents(x, weight, residual)
    # what is no tensor is refused where the other arguments are checked
    if torch.is_grad_enabled() and (x.requires_grad or getattr(weight, "requires_grad", False)
                                    or getattr(residual, "requires_grad", False)):
        y, h, rstd = _RmsNorm.apply(x, weight, residual, eps)
    else:
        y, h, rstd = _rms_forward(x, weight, eps, residual, return_rstd)
    if residual is None:
        return (y, rstd) if return_rstd else y
    return (y, h, rstd) if return_rstd else (y, h)


def rms_norm_fp8(x, weight=None, eps: float = 1e-6, residual=None, dtype=torch.float8_e4m3fn, block=128,
                 return_rstd: bool = False):
    """``rms_norm`` with its output in 8 bits: ``(q, scale)``, with a residual
    ``(q, scale, h)``, and ``rstd`` behind these with ``return_rstd``.

    ``dtype`` is ``torch.float8_e4m3fn`` or ``torch.float8_e5m2``.  ``scale``
    (float32) is the largest magnitude of a block of 128 values of a row over
    the type's largest value: shape ``x.shape[:-1] + (ceil(n / 128),)``, or
    with ``block=None`` one for the whole row, ``x.shape[:-1] + (1,)``.  ``q *
    scale`` stands for the norm, which is rounded once, from float32.  There is
    no gradient: inputs that require one are refused while gradients are
    enabled.  A training step calls it under ``torch.no_grad()`` and
    ``rms_norm_backward`` with the ``h`` (or x) and ``rstd`` it left.
    """
    if dtype not in _FP8:
        raise TypeError(f"dtype must be {' or '.join(str(d) for d in _FP8)}, got {dtype}")
    if block is not None and (isinstance(block, bool) or operator.index(block) != _BLOCK):
        raise ValueError(f"block must be {_BLOCK}, or None for whole rows, got {block}")
    eps = float(eps)
    out = _short(x, weight, eps, residual, return_rstd, _FP8[dtype], 0 if block is None else _BLOCK)
    if out is not None:
        return out
    _tensor(x, "x", _TYPES)
    _no_tangents(x, weight, residual)
    if torch.is_grad_enabled() and any(getattr(t, "requires_grad", False) for t in (x, weight, residual)):
        raise NotImplementedError("rms_norm_fp8 has no gradient: call it under torch.no_grad()")
    rows, n = _shape_2d(x, "x")
    x2, ldx, r2, ldr, sum_code, w = _rms_inputs(x, weight, residual, rows, n)
    code = _CODES[x.dtype]
    with _on(x.device):
        q = torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)
        scale = x.new_empty(x.shape[:-1] + (1 if block is None else -(-n // _BLOCK),), dtype=torch.float32)
        h = None if residual is None else torch.empty_like(residual, memory_format=torch.contiguous_format)
        rstd = x.new_empty(x.shape[:-1], dtype=torch.float32) if return_rstd else None
        _check(capi().sv_rms_norm_fp8(_ptr(x2), ldx, _ptr(r2), ldr, code, sum_code, rows, n, _ptr(w),
                                      code if w is None else _CODES[w.dtype], eps, _FP8[dtype],
                                      0 if block is None else _BLOCK, _ptr(q), n, _ptr(scale), _ptr(h), n, _ptr(rstd),
                                      _raw_stream(x.device.index)))
    return (q, scale) + (() if h is None else (h,)) + (() if rstd is None else (rstd,))


def _short_backward(*args):
    """As _short for the backward pass, with a weight."""
    if forward_ad._current_level >= 0:
        return None
    return native().rms_backward(*args)


def _rms_backward(dy, h, rstd, weight, dsum, need_dh, need_dx, need_w, param_dtype):
    _no_tangents(dy, h, rstd, weight, dsum)
    rows, n = _shape_2d(h, "h")
    w = _param(weight, "weight", dy, n) if weight is not None else None
    dy2, lddy = _rows(dy, rows, n)
    h2, ldh = _rows(h, rows, n)
    d2, ldd = _rows(dsum, rows, n) if dsum is not None else (None, n)
    rstd = _stored(rstd)
    code, sum_code = _CODES[dy.dtype], _CODES[h.dtype]
    L = capi()
    with _on(h.device):
        dh = torch.empty_like(h, memory_format=torch.contiguous_format) if need_dh else None
        dx = torch.empty_like(dy, memory_format=torch.contiguous_format) if need_dx else None
        dw = torch.empty(n, dtype=param_dtype, device=h.device) if need_w else None
        nbytes = L.sv_rms_norm_backward_workspace_size(rows, n, code, sum_code) if need_w else 0
        ws = _scratch(nbytes, h.device, "rms_norm_backward")
        _check(L.sv_rms_norm_backward(_ptr(dy2), lddy, _ptr(h2), ldh, _ptr(d2), ldd, code, sum_code, rows, n, _ptr(w),
                                      code if param_dtype is None else _CODES[param_dtype], _ptr(rstd), _ptr(dh), n,
                                      _ptr(dx), n, _ptr(dw), _ptr(ws), nbytes, _raw_stream(h.device.index)))
    return dh, dx, dw


def rms_norm_backward(dy, h, rstd, weight=None, dsum=None, *, weight_grad: bool = True, param_dtype=None):
    """Gradients ``(dh, dweight)`` of ``rms_norm`` at the rows ``h`` that were
    normed (x, or the sum it returned), for the gradient ``dy`` of its result
    and, with a residual, the gradient ``dsum`` of the sum, from the ``rstd``
    it returned.

    ``dh``, in h's type, is the gradient of x and of the residual alike.
    ``dweight`` has the weight's type (``param_dtype``, dy's type or float32,
    when there is no weight; float32 by default) and is None where not asked
    for.
    """
    if weight is not None and param_dtype in (None, getattr(weight, "dtype", None)):
        out = _short_backward(dy, h, rstd, weight, dsum, True, False, bool(weight_grad))
        if out is not None:
            return out[0], out[2]
    _tensor(dy, "dy", _TYPES)
    _tensor(h, "h", (dy.dtype, torch.float32) if dy.dtype != torch.float32 else (torch.float32,))
    _same_device(h, dy, "dy")
    if dy.shape != h.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, h {tuple(h.shape)}")
    _shape_2d(h, "h")
    _tensor(rstd, "rstd", (torch.float32,))
    _same_device(h, rstd, "rstd")
    if rstd.shape != h.shape[:-1]:
        raise ValueError(f"rstd must have shape {tuple(h.shape[:-1])}, got {tuple(rstd.shape)}")
    if dsum is not None:
        _tensor(dsum, "dsum", (h.dtype,))
        _same_device(h, dsum, "dsum")
        if dsum.shape != h.shape:
            raise ValueError(f"dsum has shape {tuple(dsum.shape)}, h {tuple(h.shape)}")
    if weight is not None:
        _tensor(weight, "weight", (dy.dtype, torch.float32))
        if param_dtype not in (None, weight.dtype):
            raise TypeError(f"param_dtype {param_dtype} differs from the weight's {weight.dtype}")
        param_dtype = weight.dtype
    elif param_dtype is None:
        param_dtype = torch.float32
    elif param_dtype not in (dy.dtype, torch.float32):
        raise TypeError(f"param_dtype must be {dy.dtype} or torch.float32, got {param_dtype}")
    dh, _, dw = _rms_backward(dy, h, rstd, weight, dsum, True, False, bool(weight_grad), param_dtype)
    return dh, dw


# ---------------------------------------------------------------- embedding

def _padding(padding_idx, vocab):
    if padding_idx is None:
        return -1
    padding_idx = operator.index(padding_idx)
    if not 0 <= padding_idx < vocab:
        raise ValueError(f"padding_idx {padding_idx} outside [0, {vocab})")
    return padding_idx


def _lookup(ids, table, scale):
    vocab, dim = table.shape
    ids1 = _stored(ids)
    t2, ldt = _rows(table, vocab, dim)
    with _on(table.device):
        out = torch.empty(ids.shape + (dim,), dtype=table.dtype, device=table.device)
        _check(capi().sv_embedding(_ptr(ids1), ids1.element_size(), ids1.numel(), _ptr(t2), _CODES[table.dtype], vocab,
                                   dim, ldt, scale, _ptr(out), dim,
                                   _raw_stream(table.device.index)))
    return out


def _lookup_backward(dy, ids, vocab, scale, padding):
    _no_tangents(dy)
    dim = dy.shape[-1]
    ids1 = _stored(ids)
    tokens = ids1.numel()
    dy2, lddy = _rows(dy, tokens, dim)
    L = capi()
    with _on(dy.device):
        grad = torch.empty(vocab, dim, dtype=dy.dtype, device=dy.device)
        nbytes = L.sv_embedding_backward_workspace_size(tokens, vocab, dim, _CODES[dy.dtype])
        ws = _scratch(nbytes, dy.device, "embedding_backward")
        _check(L.sv_embedding_backward(_ptr(dy2), lddy, _ptr(ids1), ids1.element_size(), tokens, _CODES[dy.dtype],
                                       vocab, dim, scale, padding, _ptr(grad), dim, _ptr(ws), nbytes,
                                       _raw_stream(dy.device.index)))
    return grad


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, padding):
        ctx.save_for_backward(ids)
        ctx.args = (table.shape[0], scale, padding)
        return _lookup(ids, table, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        vocab, scale, padding = ctx.args
        return None, _lookup_backward(dy, ids, vocab, scale, padding), None, None


def embedding(ids, table, scale: float = 1.0, padding_idx=None):
    """``scale * table[ids]`` for int32 or int64 ids of any shape and a table
    ``[vocab, dim]``, rounded once: shape ``ids.shape + (dim,)``.

    An id outside ``[0, vocab)`` gives a row of NaN.  ``padding_idx`` only
    concerns the gradient: its tokens take no part in it.  The table's rows may
    be strided; a table whose last dimension is not contiguous (a transposed
    one) is copied whole in every call.
    """
    _tensor(table, "table", _TYPES)
    _no_tangents(table)
    _tensor(ids, "ids", (torch.int32, torch.int64))
    _same_device(table, ids, "ids")
    if table.dim() != 2:
        raise ValueError("table must have two dimensions")
    padding = _padding(padding_idx, table.shape[0])
    if torch.is_grad_enabled() and table.requires_grad:
        return _Embedding.apply(ids, table, float(scale), padding)
    return _lookup(ids, table, float(scale))


def embedding_backward(dy, ids, num_embeddings: int, scale: float = 1.0, padding_idx=None):
    """Gradient of ``embedding``'s table, ``[num_embeddings, dim]`` in dy's
    type, for the gradient ``dy`` (``ids.shape + (dim,)``) of its result:
    each row the compensated sum of its tokens' gradients in token order,
    times ``scale``.  Ids outside the table and ``padding_idx`` take no part.
    """
    _tensor(dy, "dy", _TYPES)
    _tensor(ids, "ids", (torch.int32, torch.int64))
    _same_device(dy, ids, "ids")
    if dy.dim() != ids.dim() + 1 or dy.shape[:-1] != ids.shape:
        raise ValueError(f"dy must have shape {tuple(ids.shape)} + (dim,), got {tuple(dy.shape)}")
    num_embeddings = operator.index(num_embeddings)
    if num_embeddings < 0:
        raise ValueError("num_embeddings must be >= 0")
    return _lookup_backward(dy, ids, num_embeddings, float(scale), _padding(padding_idx, num_embeddings))
