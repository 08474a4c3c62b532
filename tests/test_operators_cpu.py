"""CPU checks of the linear layer's, the sampling's and the gradients' C ABI and bindings: exported names, argument
checks, workspace sizes, quick returns, and the references' own plants.  No call here launches work."""
import ctypes
import math
import os
import re
import types

import pytest
import torch

import fp32_gemm_05_amd as sg
from fp32_gemm_05_amd import grads, linear, sample, vocab
import linear_reference
import sample_reference

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 24  # an aligned address that is never read
MODULES = {"linear": linear, "sample": sample, "grads": grads}


@pytest.mark.parametrize("header", MODULES)
def test_header_declares_and_library_exports(header):
    module = MODULES[header]
    text = open(os.path.join(ROOT, "include", header + ".h")).read()
    names = re.findall(r"SGEMM_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert sorted(names) == sorted(module._NAMES)
    lib = ctypes.CDLL(sg.library_path())
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for n in names:
        assert hasattr(lib, n), n
        body = re.search(r"\b%s\s*\(([^)]*)\)" % n, code).group(1)
        assert [re.sub(r"[\s\*]", " ", a).split()[-1] for a in body.split(",")] == module._NAMES[n], n


T, N, H, V = 100, 1000, 64, 5000


def call(module, name, **over):
    """A valid call at made-up addresses but for `over`; returns its code."""
    args = {"dtype": 0, "out_dtype": 0, "T": T, "N": N, "H": H, "V": V, "X": A, "ldx": H, "W": 2 * A, "ldw": H, "bias": 3 * A,
            "residual": 4 * A, "ldr": N, "activation": 2, "Y": 5 * A, "ldy": N, "Z": 6 * A, "ldz": N, "dY": 7 * A,
            "lddy": N, "dX": 8 * A, "lddx": H, "dW": 9 * A, "lddw": H, "dbias": 10 * A, "work": 32 * A,
            "work_bytes": 1 << 40, "stream": None, "logits": A, "ld": V, "u": 2 * A, "temperature": 1.0,
            "temperatures": None, "top_k": 0, "top_ks": None, "top_p": 1.0, "top_ps": None, "min_p": 0.0, "min_ps": None,
            "token": 3 * A}
    args.update(over)
    return module._library[name](*[args[n] for n in module._NAMES[name]])


LINEAR = [("dtype", 2), ("dtype", -1), ("T", -1), ("T", (1 << 24) + 1), ("N", 0), ("N", (1 << 21) + 1), ("H", 0),
          ("H", (1 << 20) + 1), ("ldx", H - 1), ("ldw", H - 1), ("activation", 5), ("activation", -1), ("X", None),
          ("X", A + 2), ("W", None), ("W", 2 * A + 1), ("work", None), ("work", 32 * A + 8), ("work_bytes", 100)]
FORWARD = [("out_dtype", 1), ("out_dtype", 2), ("bias", 3 * A + 2), ("residual", 4 * A + 2), ("ldr", N - 1), ("Y", None),
           ("Y", 5 * A + 2), ("Y", A), ("Y", 2 * A + 4), ("Y", 3 * A), ("Y", 4 * A), ("ldy", N - 1), ("Z", 5 * A), ("Z", A),
           ("Z", 4 * A + 400), ("ldz", N - 1)]
GRADIENT = [("dY", None), ("lddy", N - 1), ("Z", None), ("Z", 6 * A + 1), ("ldz", N - 1), ("dX", A), ("dX", 7 * A), ("dX", 8 * A + 2),
            ("lddx", H - 1), ("dW", 8 * A), ("dW", 2 * A), ("lddw", H - 1), ("dbias", 9 * A), ("dbias", 7 * A),
            ("dbias", 6 * A), ("dbias", 10 * A + 2)]


@pytest.mark.parametrize("name,bad", [("linear_act", b) for b in LINEAR + FORWARD] + [("linear_act_grad", b) for b in LINEAR + GRADIENT])
def test_linear_refusals_name_the_argument(name, bad):
    arg, value = bad
    rc = call(linear, name, **{arg: value})
    assert rc < 0 and linear._NAMES[name][-rc - 1] == arg, (name, bad, rc)


def test_linear_sizes_that_do_not_fit_a_grid():
    f = linear._library["linear_workspace"]
    assert f(0, 0, 1 << 20, 1 << 16, 64) == -4 and f(0, 0, 1 << 20, 1 << 10, 1 << 16) == -5
    assert f(0, 0, 1 << 20, 1 << 15, 64) > 0
    for bad, code in (((2, 0, 1, 1, 1), -1), ((0, 0, -1, 1, 1), -3), ((0, 0, 1, 0, 1), -4), ((0, 0, 1, 1, 0), -5)):
        assert f(*bad) == code
    for dtype in (0, 1):
        for sizes in ((1, 1, 1), (64, 500, 8000), (65, 3, 5), (3000, 2000, 1000)):
            assert f(dtype, 0, *sizes) >= 0 and f(dtype, 1, *sizes) > 0
    with pytest.raises(sg.SgemmArgumentError) as e:
        sg.linear_workspace(torch.float32, False, 2 ** 32 + 5, 10, 4)
    assert e.value.code == -3


def test_linear_quick_returns():
    assert call(linear, "linear_act", T=0, X=None, W=None, Y=None, work=None, work_bytes=0) == 0
    assert call(linear, "linear_act_grad", dX=None, dW=None, dbias=None, work=None) == 0
    # nothing to set to zero
    assert call(linear, "linear_act_grad", T=0, dW=None, dbias=None, X=None, dY=None, Z=None, work=None, work_bytes=0) == 0


SAMPLE = [("dtype", 2), ("T", -1), ("T", (1 << 21) + 1), ("V", 0), ("V", (1 << 23) + 1), ("ld", V - 1), ("logits", None),
          ("logits", A + 2), ("u", None), ("temperature", -1.0), ("temperature", math.nan), ("temperature", math.inf),
          ("top_p", math.nan), ("min_p", math.nan), ("token", None)]


@pytest.mark.parametrize("arg,value", SAMPLE)
def test_sample_refusals_name_the_argument(arg, value):
    rc = call(sample, "vocab_sample", **{arg: value})
    assert rc < 0 and sample._NAMES["vocab_sample"][-rc - 1] == arg, (arg, value, rc)


def test_sample_quick_return_and_sizes():
    assert call(sample, "vocab_sample", T=0, logits=None, u=None, token=None, work=None, work_bytes=0) == 0
    with pytest.raises(sg.SgemmArgumentError) as e:
        sg.vocab_sample_workspace(torch.float32, 1, 2 ** 32 + 7)
    assert e.value.code == -3


def table(*rows):
    flat = (ctypes.c_longlong * (7 * len(rows)))(*[v for row in rows for v in row])
    return ctypes.addressof(flat), flat


ROW = (A, 2 * A, 10, 20, 20, 20, 0)  # x, out, rows, cols, ld, ld_out, dtype


def bad(i, value, row=ROW):
    return tuple(value if j == i else v for j, v in enumerate(row))


@pytest.mark.parametrize("rows", [
    [bad(0, 0)], [bad(0, A + 2)], [bad(2, -1)], [bad(2, 1 << 31)], [bad(3, -1)], [bad(3, (1 << 40) + 1)], [bad(4, 19)],
    [bad(4, 1 << 31)], [bad(6, 2)], [bad(6, -1)], [bad(1, 0)], [bad(1, 2 * A + 1)], [bad(5, 19)], [bad(5, 1 << 31)],
    [ROW, ROW], [bad(1, A + 4)], [ROW, bad(0, 2 * A + 400)], [bad(1, A), bad(1, A)], [ROW, (3 * A, 2 * A + 799, 1, 5, 5, 5, 0)],
    [(A, A, 10, 20, 30, 40, 0)], [(A, 2 * A, 1 << 21, 1 << 20, 1 << 20, 1 << 20, 0)]])
def test_clip_refuses_tensors(rows):
    at, keep = table(*rows)
    assert grads._library["clip_grad_norm"](len(rows), at, 1.0, 1e-6, 5 * A, 6 * A, 1 << 40, None) == -2


def test_grads_refusals():
    at, keep = table(ROW)
    norm, clip, size = (grads._library[n] for n in ("grad_norm", "clip_grad_norm", "grad_workspace"))
    assert norm(-1, at, 5 * A, 6 * A, 1 << 40, None) == -1 and norm((1 << 20) + 1, at, 5 * A, 6 * A, 1 << 40, None) == -1
    assert norm(1, None, 5 * A, 6 * A, 1 << 40, None) == -2
    assert norm(1, at, None, 6 * A, 1 << 40, None) == -3
    assert norm(1, at, 5 * A, None, 1 << 40, None) == -4 and norm(1, at, 5 * A, 6 * A + 8, 1 << 40, None) == -4
    assert norm(1, at, 5 * A, 6 * A, 10, None) == -5
    for value in (-1.0, math.nan):
        assert clip(1, at, value, 1e-6, 5 * A, 6 * A, 1 << 40, None) == -3
        assert clip(1, at, 1.0, value, 5 * A, 6 * A, 1 << 40, None) == -4
    assert clip(1, at, 1.0, 1e-6, None, 6 * A, 1 << 40, None) == -5
    assert clip(1, at, 1.0, 1e-6, 5 * A, None, 1 << 40, None) == -6
    assert clip(1, at, 1.0, 1e-6, 5 * A, 6 * A, 10, None) == -7
    assert size(0, None) > 0 and size(1, at) > size(0, None)
    # of more than 2^24 pieces a grid does not hold, larger ones are taken
    at, keep = table((A, A, (1 << 31) - 1, 512, 512, 512, 1))
    assert 0 < size(1, at) < 1 << 30


def test_errors_are_the_librarys():
    with pytest.raises(sg.SgemmArgumentError, match=r"linear_act: argument 6 \(X\) is invalid") as e:
        linear._library.fail(-6, "linear_act")
    assert e.value.code == -6 and isinstance(e.value, ValueError)
    with pytest.raises(sg.SgemmLaunchError, match="hipError_t 98"):
        grads._library.fail(98, "grad_norm")


def test_host_tensors_and_types_are_refused():
    X, W = torch.zeros(4, 8), torch.zeros(10, 8)
    with pytest.raises(ValueError, match="device tensor"):
        sg.linear_act(X, W)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sg.linear_act(X.double(), W)
    with pytest.raises(ValueError, match="device tensor"):
        sg.vocab_sample(X, torch.zeros(4))
    with pytest.raises(ValueError, match="device tensor"):
        sg.grad_norm([X])
    with pytest.raises(TypeError):
        sg.grad_norm([None])
    with pytest.raises(ValueError, match="no tensors"):
        sg.clip_grad_norm([], 1.0)


@pytest.fixture
def any_device(monkeypatch):
    for module in (vocab, linear, grads):
        monkeypatch.setattr(module, "_require_device", lambda t, name: None)


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_linear_binding_refusals(any_device):
    X, W = meta(4, 8), meta(10, 8)
    for kwargs, error, match in (
            (dict(bias=meta(9)), ValueError, "10 contiguous"), (dict(bias=meta(10, dtype=torch.bfloat16)), TypeError, "bias"),
            (dict(bias=meta(20)[::2]), ValueError, "contiguous"), (dict(residual=meta(4, 9)), ValueError, "not 4 x 10"),
            (dict(residual=meta(4, 10, dtype=torch.bfloat16)), TypeError, "residual"),
            (dict(activation="tanh"), ValueError, "gelu_tanh"), (dict(out_dtype=torch.bfloat16), TypeError, "out_dtype")):
        with pytest.raises(error, match=match):
            sg.linear_act(X, W, **kwargs)
    with pytest.raises(ValueError, match="shape mismatch"):
        sg.linear_act(X, meta(10, 9))
    with pytest.raises(ValueError, match="needs Z"):
        sg.linear_act_grad(X, W, meta(4, 10), activation="silu")
    with pytest.raises(ValueError, match="none of"):
        sg.linear_act_grad(X, W, meta(4, 10), want_dx=False, want_dw=False, want_dbias=False)
    with pytest.raises(ValueError, match="row stride 0"):
        sg.linear_act_grad(X, W, meta(10).expand(4, 10))


def test_sample_binding_refusals(any_device):
    logits, u = meta(4, 8), meta(4)
    with pytest.raises(ValueError, match="values for 4"):
        sg.vocab_sample(logits, meta(5))
    with pytest.raises(TypeError, match="top_k must be a 1-D int64"):
        sg.vocab_sample(logits, u, top_k=meta(4))
    with pytest.raises(TypeError, match="temperature must be a 1-D float32"):
        sg.vocab_sample(logits, u, temperature=meta(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="no int64"):
        sg.vocab_sample(logits, u, top_k=2 ** 63)


def test_streams_of_other_devices_are_refused():
    from fp32_gemm_05_amd import _calls
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        _calls.on_stream(torch.device("cuda", 0), stream, [], lambda: None)


# --- the references see mistakes ------------------------------------------------------------------------

def problem(dtype, name, T=30, N=40, H=50):
    g = torch.Generator().manual_seed(1)
    X, W, b, R, dY = (torch.randn(*s, generator=g).to(dtype) for s in ((T, H), (N, H), (N,), (T, N), (T, N)))
    return X, W / 7, b, R, dY


@pytest.mark.parametrize("name", linear_reference.ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_reference_layer_and_its_plants(name, dtype):
    X, W, b, R, dY = problem(dtype, name)
    x, w = X.double().requires_grad_(), W.double().requires_grad_()
    c = b.double().requires_grad_()
    f = torch.nn.functional
    act = {"none": lambda t: t, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh"), "silu": f.silu}
    y = act[name](x @ w.t() + c) + R.double()
    dX, dW, db = torch.autograd.grad((y * dY.double()).sum(), (x, w, c))
    y = y.detach()
    linear_reference.check_forward(X, W, b, R, name, y.to(dtype))
    linear_reference.check_gradients(X, W, b, dY, name, dX.to(dtype), dW.to(dtype), db.to(dtype))
    for i, wrong in enumerate((y * (1 + 2.0 ** (-6 if dtype == torch.bfloat16 else -14)), torch.where(y == y[3, 4], math.nan, y), y - R.double())):
        with pytest.raises(AssertionError):
            linear_reference.check_forward(X, W, b, R, name, wrong.to(dtype))
    for i in range(3):
        got = [dX, dW, db]
        got[i] = got[i].clone()
        got[i].view(-1)[7] = math.nan
        with pytest.raises(AssertionError):
            linear_reference.check_gradients(X, W, b, dY, name, *[t.to(dtype) for t in got])
        got[i] = (dX, dW, db)[i] * 1.1
        with pytest.raises(AssertionError):
            linear_reference.check_gradients(X, W, b, dY, name, *[t.to(dtype) for t in got])


def test_reference_sampling_and_its_plants():
    row = torch.tensor([0.0, 3.0, 1.0, 3.0, -math.inf, 2.0])
    a = sample_reference.allowed
    assert a(row, 0.0, 1.0, 0, 1.0, 0.0) == {0} and a(row, 0.999, 1.0, 0, 1.0, 0.0) == {5}
    assert a(row, 0.9, 1.0, 1, 1.0, 0.0) == {1} and a(row, 0.9, 1.0, 2, 1.0, 0.0) == {3}
    assert a(row, 0.9, 0.0, 0, 1.0, 0.0) == {1} and a(row, 0.999, 1.0, 0, 0.5, 0.0) == {3}
    assert a(row, 0.999, 1.0, 0, 1.0, 0.9) == {3} and a(row, 0.999, 1.0, 0, 1.0, 2.0) == {1}
    assert a(torch.full((3,), -math.inf), 0.5, 1.0, 0, 1.0, 0.0) == {-1}
    logits, u = row[None].repeat(2, 1), torch.tensor([0.1, 0.999])
    sample_reference.check(logits, u, torch.tensor([1, 5]))
    with pytest.raises(AssertionError):
        sample_reference.check(logits, u, torch.tensor([1, 3]))
