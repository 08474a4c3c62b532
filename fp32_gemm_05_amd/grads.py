"""Tensor forms of the gradients' norm and clipping (include/grads.h): checks, allocation of the result and
workspace, and the call.  No arithmetic happens here.

    norm = grad_norm(grads)                                   # sqrt of the sum of all squares, fp32, on the device
    norm = clip_grad_norm(grads, max_norm=1.0)                # and grads *= min(1, max_norm / (norm + eps)), in place
    norm = clip_grad_norm(grads, max_norm=1.0, out=clipped)   # or into other tensors, grads left as they are

The tensors are float32 or bfloat16, mixed as they come, on one device: contiguous ones of any shape, or matrices with
unit stride along rows or columns.  The one device's work is a few launches however many there are.

``stream`` (a torch stream of the tensors' device, or a handle) is where a call runs and where its result and its
workspace are allocated; the caller orders it behind what made the tensors, which are kept until it has read and
written them.
"""
from __future__ import annotations

import array
import ctypes

import torch

from ._calls import Entries, handle_of, on_stream
from .vocab import _MOST, _TYPES, _require_device

_NAMES = {
    "grad_workspace": ["count", "tensors"],
    "grad_norm": ["count", "tensors", "norm", "work", "work_bytes", "stream"],
    "clip_grad_norm": ["count", "tensors", "max_norm", "eps", "norm", "work", "work_bytes", "stream"],
}
_KINDS = {"work_bytes": ctypes.c_longlong, **dict.fromkeys(["max_norm", "eps"], ctypes.c_float),
          **dict.fromkeys(["tensors", "norm", "work", "stream"], ctypes.c_void_p)}
_library = Entries(_NAMES, _KINDS, {"grad_workspace": ctypes.c_longlong})


def _matrix(t, flip, name):
    """Rows, columns and row stride of a matrix, or of its transpose."""
    if t.dim() == 2:
        (rows, cols), (ld, unit) = t.shape, t.stride()
        if flip:
            rows, cols, ld, unit = cols, rows, unit, ld
        if rows <= 1:
            ld = cols
        if (cols <= 1 or unit == 1) and ld >= cols:
            if rows > _MOST or ld > _MOST:
                raise ValueError(f"{name} has {rows} rows with stride {ld}: neither may be above {_MOST}")
            return rows, cols, ld
    raise ValueError(f"{name} with shape {tuple(t.shape)} and strides {t.stride()} is neither contiguous nor a matrix "
                     f"with unit stride along its rows or columns (those of out as its tensor's); pass a contiguous copy")


def _column_major(t):
    return t.dim() == 2 and t.stride(0) == 1 and t.shape[0] > 1 and t.stride(1) >= t.shape[0]


def _table(tensors, out):
    """The tensors' array for the library; a step has some hundreds of them, so each attribute is read once."""
    entries = array.array("q")
    add = entries.extend
    place = None
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"tensors[{i}] must be a torch tensor")
        kind = _TYPES.get(t.dtype)
        if kind is None:
            raise TypeError(f"tensors[{i}] must be float32 or bfloat16, not {t.dtype}")
        at = t.get_device()
        if at != place:
            _require_device(t, f"tensors[{i}]")
            if place is not None:
                raise ValueError(f"tensors[{i}] is on {t.device}, tensors[0] on {tensors[0].device}")
            place = at
        o = t
        if out is not None:
            o = out[i]
            if not isinstance(o, torch.Tensor) or o.dtype != t.dtype:
                raise TypeError(f"out[{i}] must be a {str(t.dtype).replace('torch.', '')} tensor")
            if o.shape != t.shape:
                raise ValueError(f"out[{i}] has shape {tuple(o.shape)}, tensors[{i}] {tuple(t.shape)}")
            if o.get_device() != place:
                raise ValueError(f"out[{i}] is on {o.device}, tensors[0] on {tensors[0].device}")
        if t.is_contiguous() and (o is t or o.is_contiguous()):
            n = t.numel()
            add((t.data_ptr(), o.data_ptr(), 1, n, n, n, kind))
        else:
            flip = _column_major(t if not t.is_contiguous() else o)
            rows, cols, ld = _matrix(t, flip, f"tensors[{i}]")
            add((t.data_ptr(), o.data_ptr(), rows, cols, ld, _matrix(o, flip, f"out[{i}]")[2], kind))
    return entries


def _call(name, tensors, out, stream, *settings):
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no tensors: there is no device to put a norm on")
    if out is not None:
        out = list(out)
        if len(out) != len(tensors):
            raise ValueError(f"{len(out)} outs for {len(tensors)} tensors")
    table = _table(tensors, out)
    at, count, device = table.buffer_info()[0], len(tensors), tensors[0].device
    n = _library["grad_workspace"](count, at)
    if n < 0:
        _library.fail(n, "grad_workspace")

    def body():
        norm = torch.empty((), dtype=torch.float32, device=device)
        work = torch.empty(n, dtype=torch.uint8, device=device)
        _library.call(name, count, at, *settings, norm.data_ptr(), work.data_ptr(), n, handle_of(device))
        return norm
    return on_stream(device, stream, tensors if out is None else tensors + out, body)


def grad_norm(tensors, stream=None):
    """The square root of the sum of all elements' squares, a float32 tensor without dimensions."""
    return _call("grad_norm", tensors, None, stream)


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6, out=None, stream=None):
    """Multiplies the tensors by min(1, max_norm / (norm + eps)), in place or into the tensors `out` (each of its
    tensor's shape and type); returns their norm as it was.  No autograd graph sees it."""
    return _call("clip_grad_norm", tensors, out, stream, float(max_norm), float(eps))


def grad_workspace(tensors) -> int:
    """Bytes of workspace of a call with these tensors."""
    tensors = list(tensors)
    n = _library["grad_workspace"](len(tensors), _table(tensors, None).buffer_info()[0])
    if n < 0:
        _library.fail(n, "grad_workspace")
    return n
