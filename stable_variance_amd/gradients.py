"""The norm of a model's gradients as one vector, and their clipping to a
largest norm: calls of the C ABI.

Like the rest of the binding these functions only marshal arguments: every
call runs on the current stream of the tensors' device, allocates its outputs
and scratch from torch's allocator (so it can be captured in a HIP graph) and
does not synchronise.  They take no part in autograd: gradients are values
here.
"""
from __future__ import annotations

import ctypes
from operator import attrgetter

import torch
from torch.autograd import forward_ad

from . import SvError, _check, capi, short_way as native
from .layers import _CODES, _no_tangents, _on, _raw_stream, _stored, _TYPES, _UNSUPPORTED

__all__ = ["grad_norm", "clip_grad_norm"]

_device_type = "cuda"
_kind = attrgetter("dtype", "device", "layout")


def _dense(t):
    """t fills its memory without gaps or overlaps, in some order of its
    dimensions."""
    if t.is_contiguous():
        return True
    dims = sorted((d for d in range(t.dim()) if t.shape[d] != 1), key=lambda d: -t.stride(d))
    want = t.numel()
    for d in dims:
        want //= max(t.shape[d], 1)
        if t.stride(d) != want:
            return False
    return True


def _tensors(tensors, name):
    """The tensors as a list, checked to be float32, bfloat16 or float16 and on
    one HIP device."""
    if isinstance(tensors, torch.Tensor):
        raise TypeError(f"{name} must be a list of tensors, not one tensor")
    ts = list(tensors)
    if not ts:
        raise ValueError(f"{name} holds no tensors")
    for t in ts:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must hold torch.Tensors, got {type(t).__name__}")
    kinds = set(map(_kind, ts))
    for dtype, device, layout in kinds:
        if layout != torch.strided:
            raise TypeError(f"{name} must hold strided tensors, got {layout}")
        if dtype not in _TYPES:
            raise TypeError(f"{name} must hold {' or '.join(str(d) for d in _TYPES)}, got {dtype}")
        if device.type != _device_type:
            raise ValueError(f"{name} must be on a HIP device, got {device}")
    if len({device for _, device, _ in kinds}) > 1:
        raise ValueError(f"{name} are on different devices")
    _no_tangents(*ts)
    return ts


def _arrays(ts):
    n = len(ts)
    return ((ctypes.c_void_p * n)(*[t.data_ptr() for t in ts]), (ctypes.c_int64 * n)(*[t.numel() for t in ts]),
            (ctypes.c_int * n)(*[_CODES[t.dtype] for t in ts]))


def _scratch(L, sizes, codes, n, device):
    nbytes = L.sv_grad_norm_workspace_size(sizes, codes, n)
    if nbytes == _UNSUPPORTED:
        raise SvError(5, "grad_norm: these sizes are not supported")
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def grad_norm(grads):
    """``sqrt(sum of g^2)`` over all values of a list of tensors, as a 0-d
    float32 tensor on their device.

    The tensors are float32, bfloat16 or float16, of any shapes, the types
    mixed as they come; squares and their sum are held in float64, so values
    neither overflow nor underflow.  A tensor that does not fill its memory
    densely is copied first.  The same list of sizes and types gives the same
    bits on every run.
    """
    if forward_ad._current_level < 0:
        norm = native().grad_norm(grads)  # None for other than ordinary tensors
        if norm is not None:
            return norm
    ts = _tensors(grads, "grads")
    device = ts[0].device
    ts = [t if _dense(t) and not t.is_neg() else _stored(t) for t in ts]
    L = capi()
    with _on(device):
        ptrs, sizes, codes = _arrays(ts)
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws, nbytes = _scratch(L, sizes, codes, len(ts), device)
        _check(L.sv_grad_norm(ptrs, sizes, codes, len(ts), norm.data_ptr(), ws.data_ptr(), nbytes,
                              _raw_stream(device.index)))
    return norm


def clip_grad_norm(grads, max_norm: float, out=None):
    """Scales a list of tensors by ``min(1, max_norm / (norm + 1e-6))``, norm
    their ``grad_norm``: returns ``(out, norm)``, the norm that they had.

    ``out`` is a list of tensors of the same shapes and types (new ones by
    default); ``out=grads`` scales in place, as does an entry of ``out`` that
    is the entry of ``grads``.  Otherwise what is written must not overlap any
    tensor of either list: contiguous tensors that do are refused (``SvError``),
    and so is one strided tensor twice (``ValueError``).  The device is not
    waited for, so a norm that is Inf or NaN raises nothing: with Inf every
    finite value becomes 0 and an Inf becomes NaN, with NaN all values do.
    ``max_norm=inf`` is no limit: nothing is scaled, unless the norm is NaN.
    """
    max_norm = float(max_norm)
    if forward_ad._current_level < 0:
        result = native().clip_grad_norm(grads, max_norm, out)  # None for other than ordinary tensors
        if result is not None:
            return result
    ts = _tensors(grads, "grads")
    device = ts[0].device
    if out is None:
        with _on(device):
            outs = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in ts]
    else:
        outs = ts if out is grads else _tensors(out, "out")
        if len(outs) != len(ts):
            raise ValueError(f"out holds {len(outs)} tensors, grads {len(ts)}")
        for t, o in zip(ts, outs):
            if t is not o and (t.shape != o.shape or t.dtype != o.dtype or t.device != o.device):
                raise ValueError(f"out has a {o.dtype} tensor of shape {tuple(o.shape)} on {o.device} for a {t.dtype} "
                                 f"one of shape {tuple(t.shape)} on {t.device}")
        if torch.is_grad_enabled() and any(o.requires_grad for o in outs):
            raise ValueError("an out tensor requires a gradient: it cannot be written while gradients are enabled")
    L = capi()
    with _on(device):
        src, dst, back = [], [], []
        for t, o in zip(ts, outs):
            plain = not t.is_neg()
            if t is o and plain and _dense(t):
                src.append(t)
                dst.append(t)
                continue
            # both in one order in memory; what is not goes through a copy
            s = t if plain and t.is_contiguous() else _stored(t)
            d = o
            if o.is_neg() or not o.is_contiguous():
                if any(o.stride(i) == 0 and o.shape[i] > 1 for i in range(o.dim())):
                    raise ValueError("an out tensor has one place in memory for several values")
                d = torch.empty_like(s)
                back.append((o, d))
            src.append(s)
            dst.append(d)
        if len({(o.data_ptr(), o.shape, o.stride()) for o, _ in back}) < len(back):
            raise ValueError("out holds a tensor twice")
        ptrs, sizes, codes = _arrays(src)
        out_ptrs = (ctypes.c_void_p * len(dst))(*[d.data_ptr() for d in dst])
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws, nbytes = _scratch(L, sizes, codes, len(src), device)
        _check(L.sv_clip_grad_norm(ptrs, out_ptrs, sizes, codes, len(src), max_norm, norm.data_ptr(), ws.data_ptr(),
                                   nbytes, _raw_stream(device.index)))
        for o, d in back:
            o.detach().copy_(d)
        written = [o for o in outs if not o.is_inference()]
        if out is not None and written:
            torch.autograd.graph.increment_version(written)
    return outs, norm
