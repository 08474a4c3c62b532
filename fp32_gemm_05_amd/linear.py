"""Tensor forms of the linear layer with an epilogue (include/linear.h): checks, allocation of results and
workspace, and the call.  No arithmetic happens here.

    Y = linear_act(X, W, bias, residual, activation="gelu")        # act(X @ W.T + bias) + residual
    Y, Z = linear_act(..., keep=True)                              # Z = X @ W.T + bias, for the gradient
    dX, dW, dbias = linear_act_grad(X, W, dY, Z, activation="gelu")

X (T x H) and W (N x H) are both float32 or both bfloat16, row-major with any row stride (a contiguous copy is
asked for where rows overlap); bias (N) and residual (T x N) are of the same type, but the residual of Y's with
``out_dtype=torch.float32`` beside bfloat16 operands.  ``activation`` is one of "none", "relu", "gelu",
"gelu_tanh", "silu".  ``linear_layer`` is the same layer for torch's autograd; the functions above are no part of it.

``stream`` (a torch stream of X's device, or a handle) is where a call runs and where its results and its
workspace are allocated; the caller orders it behind what made the operands, which are kept until it
has read them.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._calls import Entries, handle_of, on_stream
from .vocab import _MOST, _TYPES, _matrix, _require_device

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_NAMES = {
    "linear_workspace": ["dtype", "grad", "T", "N", "H"],
    "linear_act": ["dtype", "out_dtype", "T", "N", "H", "X", "ldx", "W", "ldw", "bias", "residual", "ldr", "activation",
                   "Y", "ldy", "Z", "ldz", "work", "work_bytes", "stream"],
    "linear_act_grad": ["dtype", "T", "N", "H", "X", "ldx", "W", "ldw", "dY", "lddy", "Z", "ldz", "activation", "dX",
                        "lddx", "dW", "lddw", "dbias", "work", "work_bytes", "stream"],
}
_KINDS = {"work_bytes": ctypes.c_longlong,
          **dict.fromkeys(["X", "W", "bias", "residual", "Y", "Z", "dY", "dX", "dW", "dbias", "work", "stream"],
                          ctypes.c_void_p)}
_library = Entries(_NAMES, _KINDS, {"linear_workspace": ctypes.c_longlong})


def linear_workspace(dtype, grad: bool, T: int, N: int, H: int) -> int:
    """Bytes of workspace of a call of linear_act (grad False) or linear_act_grad."""
    return _workspace(dtype, bool(grad), int(T), int(N), int(H))


@functools.lru_cache(maxsize=256)
def _workspace(dtype, grad, T, N, H):
    for i, n in enumerate((T, N, H)):
        if abs(n) > _MOST:
            _library.fail(-3 - i, "linear_workspace")
    n = _library["linear_workspace"](_TYPES[dtype], grad, T, N, H)
    if n < 0:
        _library.fail(n, "linear_workspace")
    return n


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, not {name!r}")
    return ACTIVATIONS[name]


def _of(t, name, rows, cols, dtype, device):
    """The address and row stride of a rows x cols matrix of `dtype` on `device`."""
    r, c, ld = _matrix(t, name, dtype)
    if (r, c) != (rows, cols):
        raise ValueError(f"{name} is {r} x {c}, not {rows} x {cols}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, X on {device}")
    return t.data_ptr(), ld


def _operands(X, W):
    T, H, ldx = _matrix(X, "X")
    N, h, ldw = _matrix(W, "W", X.dtype)
    if h != H:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
    if N < 1 or H < 1:
        raise ValueError(f"W {tuple(W.shape)} has no element")
    if W.device != X.device:
        raise ValueError(f"W is on {W.device}, X on {X.device}")
    return T, N, H, (X.data_ptr(), ldx, W.data_ptr(), ldw)


def _work(grad, dtype, T, N, H, device):
    n = _workspace(dtype, grad, T, N, H)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def linear_act(X, W, bias=None, residual=None, activation: str = "none", out_dtype=None, keep: bool = False, stream=None):
    """act(X @ W.T + bias) + residual in X's type, or in float32 (out_dtype, beside bfloat16 operands); with
    ``keep`` also X @ W.T + bias in X's type, which linear_act_grad takes: (Y, Z)."""
    T, N, H, matrices = _operands(X, W)
    dtype, device = X.dtype, X.device
    act = _activation(activation)
    out_dtype = dtype if out_dtype is None else out_dtype
    if out_dtype != dtype and out_dtype != torch.float32:
        raise TypeError(f"out_dtype must be float32 or X's type, not {out_dtype}")
    at_bias = None
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype != dtype or bias.dim() != 1:
            raise TypeError(f"bias must be a 1-D {str(dtype).replace('torch.', '')} tensor")
        _require_device(bias, "bias")
        if bias.shape[0] != N or (N > 1 and bias.stride(0) != 1):
            raise ValueError(f"bias must be {N} contiguous values")
        if bias.device != device:
            raise ValueError(f"bias is on {bias.device}, X on {device}")
        at_bias = bias.data_ptr()
    at_residual, ldr = (None, N) if residual is None else _of(residual, "residual", T, N, out_dtype, device)

    def body():
        Y = torch.empty((T, N), dtype=out_dtype, device=device)
        Z = torch.empty((T, N), dtype=dtype, device=device) if keep else None
        work = _work(False, dtype, T, N, H, device)
        _library.call("linear_act", _TYPES[dtype], _TYPES[out_dtype], T, N, H, *matrices, at_bias, at_residual, ldr, act,
                      Y.data_ptr(), N, Z.data_ptr() if keep else None, N, None if work is None else work.data_ptr(),
                      0 if work is None else work.numel(), handle_of(device))
        return (Y, Z) if keep else Y
    return on_stream(device, stream, (X, W, bias, residual), body)


def linear_act_grad(X, W, dY, Z=None, activation: str = "none", want_dx: bool = True, want_dw: bool = True,
                    want_dbias: bool = True, stream=None):
    """Gradients (dX, dW, dbias) of sum(dY * Y), in X's type, from the Z that linear_act kept (None without an
    activation); one that is not wanted is None and costs no product.  The residual's gradient is dY."""
    T, N, H, matrices = _operands(X, W)
    dtype, device = X.dtype, X.device
    act = _activation(activation)
    at_dy, lddy = _of(dY, "dY", T, N, dtype, device)
    at_z, ldz = None, N
    if act:
        if Z is None:
            raise ValueError(f"the gradient of {activation} needs Z (keep=True)")
        at_z, ldz = _of(Z, "Z", T, N, dtype, device)
    if not (want_dx or want_dw or want_dbias):
        raise ValueError("none of dX, dW and dbias is wanted")

    def body():
        dX = torch.empty((T, H), dtype=dtype, device=device) if want_dx else None
        dW = torch.empty((N, H), dtype=dtype, device=device) if want_dw else None
        dbias = torch.empty(N, dtype=dtype, device=device) if want_dbias else None
        work = _work(True, dtype, T, N, H, device)
        _library.call("linear_act_grad", _TYPES[dtype], T, N, H, *matrices, at_dy, lddy, at_z, ldz, act,
                      dX.data_ptr() if want_dx else None, H, dW.data_ptr() if want_dw else None, H,
                      dbias.data_ptr() if want_dbias else None, None if work is None else work.data_ptr(),
                      0 if work is None else work.numel(), handle_of(device))
        return dX, dW, dbias
    return on_stream(device, stream, (X, W, dY, Z), body)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, bias, residual, activation):
        keep = activation != "none" and any(ctx.needs_input_grad[:3])
        Y = linear_act(X, W, bias, residual, activation, keep=keep)
        Y, Z = Y if keep else (Y, None)
        ctx.save_for_backward(X, W, Z)
        ctx.activation = activation
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        X, W, Z = ctx.saved_tensors
        want = ctx.needs_input_grad
        dX = dW = dbias = None
        if any(want[:3]):
            dX, dW, dbias = linear_act_grad(X, W, dY.contiguous(), Z, ctx.activation, want_dx=want[0], want_dw=want[1],
                                            want_dbias=want[2])
        return dX, dW, dbias, dY if want[3] else None, None


def linear_layer(X, W, bias=None, residual=None, activation: str = "none"):
    """linear_act's Y, differentiable with respect to X, W, bias and residual.

    A backward pass may be captured into a graph, with torch.autograd.grad, or with leaves that no eager graph still
    holds: torch's own accumulation of gradients of such leaves ends the process in a capture."""
    return _Linear.apply(X, W, bias, residual, activation)
