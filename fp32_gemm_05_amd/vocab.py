"""Tensor forms of the vocabulary-head operators (include/vocab.h): checks, allocation of results and
workspace, and the call.  No arithmetic happens here.

    loss, lse = vocab_ce(X, W, target)                                  # per token, fp32
    dX, dW = vocab_ce_grad(X, W, target, lse, dloss)
    loss, lse, picked = vocab_distill(X, W, index, teacher)
    dX, dW = vocab_distill_grad(X, W, index, teacher, lse, picked, dloss)

X (T x H) and W (V x H) are both float32 or both bfloat16, row-major with any row stride (a
contiguous copy is asked for where rows overlap).  ``vocab_cross_entropy`` and
``vocab_distillation`` are the same operators for torch's autograd, which gives gradients of the losses
alone; the four functions above are no part of it: their results carry no gradient, also where X or W
requires one.

``stream`` (a torch stream of X's device, or a handle) is where a call runs and where its results and its
workspace are allocated; the caller orders it behind what made the operands, which are kept until it
has read them.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import SgemmArgumentError, SgemmError, SgemmLaunchError, _require_device, load_library

_TYPES = {torch.float32: 0, torch.bfloat16: 1}

_HEAD = ["dtype", "T", "V", "H"]
_MATRICES = ["X", "ldx", "W", "ldw"]
_OUT = ["dX", "lddx", "dW", "lddw", "work", "work_bytes", "stream"]
_NAMES = {
    "vocab_workspace": ["dtype", "grad", "T", "V", "H", "K"],
    "vocab_ce": _HEAD + ["alpha"] + _MATRICES + ["target", "ignore_index", "loss", "lse", "work", "work_bytes",
                                                 "stream"],
    "vocab_ce_grad": _HEAD + ["alpha"] + _MATRICES + ["target", "ignore_index", "lse", "dloss"] + _OUT,
    "vocab_distill": _HEAD + ["K", "alpha", "teacher_alpha"] + _MATRICES + [
        "index", "ldi", "teacher", "ldt", "loss", "lse", "picked", "work", "work_bytes", "stream"],
    "vocab_distill_grad": _HEAD + ["K", "alpha", "teacher_alpha"] + _MATRICES + [
        "index", "ldi", "teacher", "ldt", "lse", "picked", "dloss"] + _OUT,
}
_KINDS = {"alpha": ctypes.c_float, "teacher_alpha": ctypes.c_float, "ignore_index": ctypes.c_longlong,
          "work_bytes": ctypes.c_longlong,
          **dict.fromkeys(["X", "W", "target", "index", "teacher", "loss", "lse", "picked", "dloss", "dX", "dW",
                           "work", "stream"], ctypes.c_void_p)}
_entries = {}
_MOST = 2 ** 31 - 1  # of a size or a row stride: ctypes would pass on the low 32 bits of a larger one


def _entry(name):
    if name not in _entries:
        f = getattr(load_library(), name)
        f.argtypes = [_KINDS.get(a, ctypes.c_int) for a in _NAMES[name]]
        f.restype = ctypes.c_longlong if name == "vocab_workspace" else ctypes.c_int
        _entries[name] = f
    return _entries[name]


def _raise(code, name):
    names = _NAMES[name]
    if code < 0:
        what = f"argument {-code} ({names[-code - 1] if -code <= len(names) else '?'}) is invalid"
    else:
        what = f"kernel launch failed with hipError_t {code}"
    error = SgemmError.__new__(SgemmArgumentError if code < 0 else SgemmLaunchError)
    RuntimeError.__init__(error, f"{name}: {what}")
    error.code = code
    raise error


def vocab_workspace(dtype, grad: bool, T: int, V: int, H: int, K: int = 0) -> int:
    """Bytes of workspace of a call (K = 0: cross entropy, else the teacher's entries per token)."""
    return _workspace(dtype, bool(grad), int(T), int(V), int(H), int(K))


@functools.lru_cache(maxsize=256)
def _workspace(dtype, grad, T, V, H, K):
    for i, n in enumerate((T, V, H, K)):
        if abs(n) > _MOST:
            _raise(-3 - i, "vocab_workspace")
    n = _entry("vocab_workspace")(_TYPES[dtype], grad, T, V, H, K)
    if n < 0:
        _raise(n, "vocab_workspace")
    return n


# The checks and calls below take about as long as two kernel launches, which is what a small problem
# takes in all: attributes are read once, and no stream or device context is entered without need.

def _matrix(t, name, dtype=None):
    """Checks a 2-D device tensor with unit column stride; returns (rows, columns, leading dimension)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != 2 or (t.dtype not in _TYPES if dtype is None else t.dtype != dtype):
        want = "float32 or bfloat16" if dtype is None else str(dtype).replace("torch.", "")
        raise TypeError(f"{name} must be a 2-D {want} tensor")
    _require_device(t, name)
    rows, cols = t.shape
    ld, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if rows <= 1 or cols == 0:
        ld = cols if cols > 1 else 1  # one row, or no element: no stride is addressed
    elif ld < cols:
        raise ValueError(f"{name} has row stride {ld} below its row length {cols} "
                         f"(a broadcast or overlapping view); pass a contiguous copy")
    if rows > _MOST or ld > _MOST:
        raise ValueError(f"{name} has {rows} rows with stride {ld}: neither may be above {_MOST}")
    return rows, cols, ld


def _ignored(index):
    index = int(index)
    if not -2 ** 63 <= index < 2 ** 63:
        raise ValueError(f"ignore_index {index} is no int64")
    return index


def _vector(t, name, dtype, n):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype or t.dim() != 1:
        raise TypeError(f"{name} must be a 1-D {str(dtype).replace('torch.', '')} tensor")
    _require_device(t, name)
    if t.shape[0] != n:
        raise ValueError(f"{name} has {t.shape[0]} values for {n} tokens")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


# torch.cuda.current_stream makes a Stream object first, 20 times the time of the handle alone
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_device(stream, device):
    """The torch stream of a handle or stream, which has to be `device`'s."""
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, X on {device}")
    return stream


class _Problem:
    """The checked operands that every call has, and what they share."""

    __slots__ = ("T", "V", "H", "K", "dtype", "device", "head", "matrices", "alpha", "context", "stream", "read")

    def __init__(self, X, W, alpha, stream, entries=0):
        self.T, self.H, ldx = _matrix(X, "X")
        self.dtype = X.dtype
        self.V, H, ldw = _matrix(W, "W", self.dtype)
        if self.H != H:
            raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
        if self.V < 1 or H < 1:
            raise ValueError(f"W {tuple(W.shape)} has no element")
        self.K = entries
        self.device = X.device
        self.head = (_TYPES[self.dtype], self.T, self.V, H)
        self.matrices = (X.data_ptr(), ldx, W.data_ptr(), ldw)
        self.alpha = float(alpha)
        self.read = [X]
        self.same_device(W, "W")
        # results and workspace are allocated on the stream that uses them; the operands are told of it, so
        # that their memory is not given out again before it has read them
        self.context = self.stream = None
        if stream is not None:
            self.stream = _on_device(stream, self.device)
            self.context = torch.cuda.stream(self.stream)
        elif self.device.index != torch.cuda.current_device():
            self.context = torch.cuda.device(self.device)

    def same_device(self, t, name):
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, X on {self.device}")
        self.read.append(t)

    def vector(self, t, name, dtype=torch.float32):
        _vector(t, name, dtype, self.T)
        self.same_device(t, name)

    def run(self, body):
        if self.context is None:
            return body()
        with self.context:
            try:
                return body()
            finally:
                if self.stream is not None:
                    for t in self.read:
                        t.record_stream(self.stream)

    def new(self, *shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, grad):
        """Kept by the caller until the call has enqueued its work; the stream's own pool takes it back."""
        n = vocab_workspace(self.dtype, grad, self.T, self.V, self.H, self.K)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def call(self, name, work, *args):
        rc = (_entries.get(name) or _entry(name))(*args, work.data_ptr(), work.numel(),
                                                  _current_handle(self.device.index))
        if rc != 0:
            _raise(rc, name)


def vocab_ce(X, W, target, alpha: float = 1.0, ignore_index: int = -100, stream=None):
    """Per-token cross entropy of alpha * X @ W.T against target (int64): (loss, lse), both fp32.

    Tokens whose target is ignore_index have loss 0 and lse 0; a target outside the vocabulary
    gives NaN."""
    p = _Problem(X, W, alpha, stream)
    p.vector(target, "target", torch.int64)

    def body():
        loss, lse = p.new(p.T), p.new(p.T)
        p.call("vocab_ce", p.workspace(False), *p.head, p.alpha, *p.matrices, target.data_ptr(), _ignored(ignore_index),
               loss.data_ptr(), lse.data_ptr())
        return loss, lse
    return p.run(body)


def _gradients(p, want_dx, want_dw, name, *args):
    """Allocates the wanted gradients, and calls `name` with args and them."""
    if not (want_dx or want_dw):
        raise ValueError("neither dX nor dW is wanted")

    def body():
        dX = p.new(p.T, p.H, dtype=p.dtype) if want_dx else None
        dW = p.new(p.V, p.H, dtype=p.dtype) if want_dw else None
        p.call(name, p.workspace(True), *args, None if dX is None else dX.data_ptr(), p.H,
               None if dW is None else dW.data_ptr(), p.H)
        return dX, dW
    return p.run(body)


def vocab_ce_grad(X, W, target, lse, dloss, alpha: float = 1.0, ignore_index: int = -100, want_dx: bool = True,
                  want_dw: bool = True, stream=None):
    """Gradients (dX, dW) of sum(dloss * loss), from the lse of vocab_ce; one that is not wanted is None
    and costs no product."""
    p = _Problem(X, W, alpha, stream)
    p.vector(target, "target", torch.int64)
    p.vector(lse, "lse")
    p.vector(dloss, "dloss")
    return _gradients(p, want_dx, want_dw, "vocab_ce_grad", *p.head, p.alpha, *p.matrices, target.data_ptr(),
                      _ignored(ignore_index), lse.data_ptr(), dloss.data_ptr())


def _distill(X, W, index, teacher, alpha, stream):
    rows, k, ldi = _matrix(index, "index", torch.int64)
    rows_t, k_t, ldt = _matrix(teacher, "teacher", torch.float32)
    if (rows, k) != (rows_t, k_t):
        raise ValueError(f"shape mismatch: index {tuple(index.shape)}, teacher {tuple(teacher.shape)}")
    if k < 1:
        raise ValueError("index has no entry")
    p = _Problem(X, W, alpha, stream, k)
    if rows != p.T:
        raise ValueError(f"index has {rows} rows for {p.T} tokens")
    p.same_device(index, "index")
    p.same_device(teacher, "teacher")
    return p, (index.data_ptr(), ldi, teacher.data_ptr(), ldt)


def vocab_distill(X, W, index, teacher, alpha: float = 1.0, teacher_alpha: float = 1.0, stream=None):
    """Per-token divergence of softmax(alpha * X @ W.T) from a teacher's top logits: (loss, lse, picked).

    index (T x K, int64) names vocabulary rows, teacher (T x K, fp32) their logits; an index < 0 is
    no entry, and a token without entries has loss 0.  picked (T x K) holds the student's logits at
    the entries, which the gradient takes back."""
    p, entries = _distill(X, W, index, teacher, alpha, stream)

    def body():
        loss, lse, picked = p.new(p.T), p.new(p.T), p.new(p.T, p.K)
        p.call("vocab_distill", p.workspace(False), *p.head, p.K, p.alpha, float(teacher_alpha), *p.matrices, *entries,
               loss.data_ptr(), lse.data_ptr(), picked.data_ptr())
        return loss, lse, picked
    return p.run(body)


def vocab_distill_grad(X, W, index, teacher, lse, picked, dloss, alpha: float = 1.0, teacher_alpha: float = 1.0,
                       want_dx: bool = True, want_dw: bool = True, stream=None):
    """Gradients (dX, dW) of sum(dloss * loss), from the lse and picked of vocab_distill."""
    p, entries = _distill(X, W, index, teacher, alpha, stream)
    p.vector(lse, "lse")
    p.vector(dloss, "dloss")
    if _matrix(picked, "picked", torch.float32) != (p.T, p.K, p.K):
        raise ValueError("picked must be the contiguous T x K tensor of vocab_distill")
    p.same_device(picked, "picked")
    return _gradients(p, want_dx, want_dw, "vocab_distill_grad", *p.head, p.K, p.alpha, float(teacher_alpha),
                      *p.matrices, *entries, lse.data_ptr(), picked.data_ptr(), dloss.data_ptr())


class _CrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, target, alpha, ignore_index):
        loss, lse = vocab_ce(X, W, target, alpha, ignore_index)
        ctx.save_for_backward(X, W, target, lse)
        ctx.args = alpha, ignore_index
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        X, W, target, lse = ctx.saved_tensors
        dX, dW = vocab_ce_grad(X, W, target, lse, dloss.contiguous(), *ctx.args, want_dx=ctx.needs_input_grad[0],
                               want_dw=ctx.needs_input_grad[1])
        return dX, dW, None, None, None


class _Distillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, index, teacher, alpha, teacher_alpha):
        loss, lse, picked = vocab_distill(X, W, index, teacher, alpha, teacher_alpha)
        ctx.save_for_backward(X, W, index, teacher, lse, picked)
        ctx.args = alpha, teacher_alpha
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        X, W, index, teacher, lse, picked = ctx.saved_tensors
        dX, dW = vocab_distill_grad(X, W, index, teacher, lse, picked, dloss.contiguous(), *ctx.args,
                                    want_dx=ctx.needs_input_grad[0], want_dw=ctx.needs_input_grad[1])
        return dX, dW, None, None, None, None


def vocab_cross_entropy(X, W, target, alpha: float = 1.0, ignore_index: int = -100):
    """vocab_ce's loss per token, differentiable with respect to X and W."""
    return _CrossEntropy.apply(X, W, target, alpha, ignore_index)


def vocab_distillation(X, W, index, teacher, alpha: float = 1.0, teacher_alpha: float = 1.0):
    """vocab_distill's loss per token, differentiable with respect to X and W (not the teacher)."""
    return _Distillation.apply(X, W, index, teacher, alpha, teacher_alpha)
