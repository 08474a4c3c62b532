"""What the tensor forms of the operators share: entry points of the library by their argument names, its
errors, and the stream and device that a call runs on."""
from __future__ import annotations

import ctypes

import torch

from ._binding import SgemmArgumentError, SgemmError, SgemmLaunchError, load_library
from .vocab import _current_handle, _on_device


class Entries:
    """The library's functions named in `names` (name -> argument names); `kinds` gives the ctypes kind of an
    argument (int where it does not), `results` that of a result."""

    def __init__(self, names, kinds, results=None):
        self.names, self.kinds, self.results = names, kinds, results or {}
        self.found = {}

    def __getitem__(self, name):
        f = self.found.get(name)
        if f is None:
            f = getattr(load_library(), name)
            f.argtypes = [self.kinds.get(a, ctypes.c_int) for a in self.names[name]]
            f.restype = self.results.get(name, ctypes.c_int)
            self.found[name] = f
        return f

    def fail(self, code, name):
        """Raises the library's error for a code other than 0."""
        names = self.names[name]
        if code < 0:
            what = f"argument {-code} ({names[-code - 1] if -code <= len(names) else '?'}) is invalid"
        else:
            what = f"kernel launch failed with hipError_t {code}"
        error = SgemmError.__new__(SgemmArgumentError if code < 0 else SgemmLaunchError)
        RuntimeError.__init__(error, f"{name}: {what}")
        error.code = code
        raise error

    def call(self, name, *args):
        rc = self[name](*args)
        if rc != 0:
            self.fail(rc, name)


def handle_of(device):
    return _current_handle(device.index)


def on_stream(device, stream, read, body):
    """body() with `device` current, on `stream` (a torch stream of that device, or a handle) where one is given:
    results and workspaces are then allocated on it, and the tensors `read` are kept until it has read them."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return body()
        with torch.cuda.device(device):
            return body()
    stream = _on_device(stream, device)
    with torch.cuda.stream(stream):
        try:
            return body()
        finally:
            for t in read:
                if t is not None:
                    t.record_stream(stream)
