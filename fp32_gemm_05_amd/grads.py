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
    shape, strides = t.shape, t.stride()
    if len(shape) == 2:
        (rows, cols), (ld, unit) = (shape, strides) if not flip else (shape[::-1], strides[::-1])
        if rows <= 1:
            ld = cols
        if (unit == 1 or cols <= 1) and ld >= cols:
            if rows > _MOST or ld > _MOST:
                raise ValueError(f"{name} has {rows} rows with stride {ld}: neither may be above {_MOST}")
            return rows, cols, ld
    raise ValueError(f"{name} with shape {tuple(shape)} and strides {strides} is neither contiguous nor a matrix "
                     f"with unit stride along its rows or columns (those of out as its tensor's); pass a contiguous copy")


def _column_major(t):
    strides = t.stride()
    return len(strides) == 2 and strides[0] == 1 and t.shape[0] > 1 and strides[1] >= t.shape[0]


def _kinds(tensors, name):
    """The types, of tensors of one device."""
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{i}] must be a torch tensor")
    try:
        kinds = [_TYPES[t.dtype] for t in tensors]
    except KeyError:
        i = next(i for i, t in enumerate(tensors) if t.dtype not in _TYPES)
        raise TypeError(f"{name}[{i}] must be float32 or bfloat16, not {tensors[i].dtype}") from None
    places = [t.get_device() for t in tensors]
    first = places[0]
    if first < 0 or places.count(first) != len(places):
        for i, t in enumerate(tensors):
            _require_device(t, f"{name}[{i}]")
            if t.get_device() != first:
                raise ValueError(f"{name}[{i}] is on {t.device}, {name}[0] on {tensors[0].device}")
    return kinds


def _table(tensors, out):
    """The tensors' array for the library.  A step has some hundreds of them, and the work on the device takes about
    half a microsecond each: their attributes are read column by column."""
    n, kinds = len(tensors), _kinds(tensors, "tensors")
    outs = tensors if out is None else out
    if out is not None:
        if _kinds(out, "out") != kinds:
            i = next(i for i in range(n) if out[i].dtype != tensors[i].dtype)
            raise TypeError(f"out[{i}] must be a {str(tensors[i].dtype).replace('torch.', '')} tensor")
        if out[0].get_device() != tensors[0].get_device():
            raise ValueError(f"out[0] is on {out[0].device}, tensors[0] on {tensors[0].device}")
        if [t.shape for t in out] != [t.shape for t in tensors]:
            i = next(i for i in range(n) if out[i].shape != tensors[i].shape)
            raise ValueError(f"out[{i}] has shape {tuple(out[i].shape)}, tensors[{i}] {tuple(tensors[i].shape)}")
    sizes = array.array("q", [t.numel() for t in tensors])
    entries = array.array("q", bytes(56 * n))
    entries[0::7] = array.array("q", [t.data_ptr() for t in tensors])
    entries[1::7] = entries[0::7] if out is None else array.array("q", [t.data_ptr() for t in out])
    entries[2::7] = array.array("q", [1]) * n
    for column in (3, 4, 5):
        entries[column::7] = sizes
    entries[6::7] = array.array("q", kinds)
    whole = [t.is_contiguous() for t in tensors]
    whole_out = whole if out is None else [t.is_contiguous() for t in out]
    for i in range(n):
        if whole[i] and whole_out[i]:
            continue
        t, o = tensors[i], outs[i]
        flip = _column_major(o if whole[i] else t)
        rows, cols, ld = _matrix(t, flip, f"tensors[{i}]")
        at = 7 * i
        entries[at + 2], entries[at + 3], entries[at + 4] = rows, cols, ld
        if o is t:
            entries[at + 5] = ld
        else:
            entries[at + 5] = cols if whole_out[i] and not flip else _matrix(o, flip, f"out[{i}]")[2]
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
        if settings:  # clipping has written them: autograd must not take them for what it saved
            torch.autograd.graph.increment_version(tensors if out is None else out)
        return norm
    return on_stream(device, stream, tensors if out is None else tensors + out, body)


def grad_norm(tensors, stream=None):
    """The square root of the sum of all elements' squares, a float32 tensor without dimensions."""
    return _call("grad_norm", tensors, None, stream)


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6, out=None, stream=None):
    """Multiplies the tensors by min(1, max_norm / (norm + eps)), in place or into the tensors `out` (each of its
    tensor's shape and type); returns their norm as it was.  It is no part of autograd, which sees a change in place, as of
    torch's own operations: a backward pass that has saved a tensor clipped since raises an error."""
    return _call("clip_grad_norm", tensors, out, stream, float(max_norm), float(eps))


def grad_workspace(tensors) -> int:
    """Bytes of workspace of a call with these tensors."""
    tensors = list(tensors)
    n = _library["grad_workspace"](len(tensors), _table(tensors, None).buffer_info()[0])
    if n < 0:
        _library.fail(n, "grad_workspace")
    return n
