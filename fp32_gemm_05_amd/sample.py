"""Tensor form of the drawing of tokens (include/sample.h): checks, allocation of the result and workspace, and
the call.  No arithmetic happens here.

    token = vocab_sample(logits, u, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)     # int64, per row

logits (T x V) is float32 or bfloat16, row-major with any row stride, u (T, float32) random numbers in [0, 1), given by
the caller.  Each setting is one number for all rows or a tensor of T values (float32; top_k int64).

``stream`` (a torch stream of the logits' device, or a handle) is where the call runs and where its result and its
workspace are allocated; the caller orders it behind what made the operands, which are kept until it has
read them.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._calls import Entries, handle_of, on_stream
from .vocab import _MOST, _TYPES, _matrix, _vector

_NAMES = {
    "vocab_sample_workspace": ["dtype", "T", "V"],
    "vocab_sample": ["dtype", "T", "V", "logits", "ld", "u", "temperature", "temperatures", "top_k", "top_ks", "top_p",
                     "top_ps", "min_p", "min_ps", "token", "work", "work_bytes", "stream"],
}
_KINDS = {**dict.fromkeys(["temperature", "top_p", "min_p"], ctypes.c_float),
          **dict.fromkeys(["top_k", "work_bytes"], ctypes.c_longlong),
          **dict.fromkeys(["logits", "u", "temperatures", "top_ks", "top_ps", "min_ps", "token", "work", "stream"],
                          ctypes.c_void_p)}
_library = Entries(_NAMES, _KINDS, {"vocab_sample_workspace": ctypes.c_longlong})


def vocab_sample_workspace(dtype, T: int, V: int) -> int:
    """Bytes of workspace of a call."""
    return _workspace(dtype, int(T), int(V))


@functools.lru_cache(maxsize=256)
def _workspace(dtype, T, V):
    for i, n in enumerate((T, V)):
        if abs(n) > _MOST:
            _library.fail(-2 - i, "vocab_sample_workspace")
    n = _library["vocab_sample_workspace"](_TYPES[dtype], T, V)
    if n < 0:
        _library.fail(n, "vocab_sample_workspace")
    return n


def vocab_sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """One token per row of logits (int64; -1 for a row without a distribution): temperature, then top_k, top_p and
    min_p in this order, then the token up to which more than u of the probability of what stays lies, by index.

    temperature 0 takes the largest logit; top_k <= 0, top_p >= 1 and min_p <= 0 leave everything."""
    T, V, ld = _matrix(logits, "logits")
    device = logits.device
    read = [logits, u]

    def per_row(value, name, dtype):
        _vector(value, name, dtype, T)
        if value.device != device:
            raise ValueError(f"{name} is on {value.device}, logits on {device}")
        read.append(value)
        return value.data_ptr()

    at_u = per_row(u, "u", torch.float32)
    settings = []
    for value, name in ((temperature, "temperature"), (top_k, "top_k"), (top_p, "top_p"), (min_p, "min_p")):
        whole = name == "top_k"
        if isinstance(value, torch.Tensor):
            settings += [0, per_row(value, name, torch.int64 if whole else torch.float32)]
        else:
            value = int(value) if whole else float(value)
            if whole and not -2 ** 63 <= value < 2 ** 63:
                raise ValueError(f"top_k {value} is no int64")
            settings += [value, None]

    def body():
        token = torch.empty(T, dtype=torch.int64, device=device)
        n = _workspace(logits.dtype, T, V)
        work = torch.empty(n, dtype=torch.uint8, device=device) if n else None
        _library.call("vocab_sample", _TYPES[logits.dtype], T, V, logits.data_ptr(), ld, at_u, *settings, token.data_ptr(),
                      work.data_ptr() if n else None, n, handle_of(device))
        return token
    return on_stream(device, stream, read, body)
