"""CPU checks of the vocabulary-head operators' C ABI and binding: exported names, argument checks, workspace
sizes, quick returns, and the LDS layout of the tile loop against the measured pass model.  No call here
launches work."""
import ctypes
import os
import re

import pytest
import torch

import fp32_gemm_05_amd as sg
from fp32_gemm_05_amd import vocab as binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # an aligned address that is never read


def call(name, **over):
    """A valid call of `name` at made-up addresses but for `over`; returns its code."""
    T, V, H, K = 100, 1000, 64, 4
    args = {"dtype": 0, "T": T, "V": V, "H": H, "K": K, "alpha": 1.0, "teacher_alpha": 1.0, "X": A, "ldx": H,
            "W": A * 2, "ldw": H, "target": A * 3, "ignore_index": -100, "loss": A * 4, "lse": A * 5,
            "index": A * 6, "ldi": K, "teacher": A * 7, "ldt": K, "picked": A * 8, "dloss": A * 9, "dX": A * 10,
            "lddx": H, "dW": A * 11, "lddw": H, "work": A * 16, "work_bytes": 1 << 40, "stream": None}
    args.update(over)
    return binding._entry(name)(*[args[n] for n in binding._NAMES[name]])


def test_header_declares_and_library_exports():
    text = open(os.path.join(ROOT, "include", "vocab.h")).read()
    names = re.findall(r"SGEMM_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert sorted(names) == sorted(binding._NAMES)
    lib = ctypes.CDLL(sg.library_path())
    for n in names:
        assert hasattr(lib, n), n
    # the binding's argument names are the header's, in order
    for n in names:
        body = re.search(r"\b%s\s*\(([^)]*)\)" % n, re.sub(r"/\*.*?\*/", "", text, flags=re.S)).group(1)
        assert [re.sub(r"[\s\*]", " ", a).split()[-1] for a in body.split(",")] == binding._NAMES[n], n


COMMON = [("dtype", 2), ("dtype", -1), ("T", -1), ("T", (1 << 21) + 1), ("V", 0), ("V", -5), ("H", 0),
          ("H", (1 << 20) + 1), ("ldx", 63), ("ldw", 63), ("X", None), ("W", None), ("work", None), ("work", A + 8),
          ("work_bytes", 100)]
GRAD = [("lddx", 63), ("lddw", 63), ("lse", None), ("dloss", None), ("dX", A), ("dX", A * 2), ("dW", A), ("dW", A * 2),
        ("dW", A * 10 + 256)]
CE = [("target", None)]
DISTILL = [("K", 0), ("ldi", 3), ("ldt", 3), ("index", None), ("teacher", None), ("picked", None)]


@pytest.mark.parametrize("name,bad", [(n, b) for n, cases in (
    ("vocab_ce", COMMON + CE + [("loss", None), ("lse", None)]),
    ("vocab_ce_grad", COMMON + CE + GRAD),
    ("vocab_distill", COMMON + DISTILL + [("loss", None), ("lse", None)]),
    ("vocab_distill_grad", COMMON + DISTILL + GRAD)) for b in cases])
def test_refusals_name_the_argument(name, bad):
    arg, value = bad
    rc = call(name, **{arg: value})
    assert rc < 0 and binding._NAMES[name][-rc - 1] == arg, (name, bad, rc)


def test_too_many_entries():
    assert call("vocab_distill", T=1 << 20, K=1 << 11, ldi=1 << 11, ldt=1 << 11) == -5


def test_quick_returns():
    assert call("vocab_ce", T=0, X=None, target=None, loss=None, lse=None, work=None) == 0
    assert call("vocab_distill", T=0) == 0
    assert call("vocab_ce_grad", dX=None, dW=None, work=None) == 0
    assert call("vocab_distill_grad", dX=None, dW=None) == 0


def test_workspace():
    f = binding.vocab_workspace
    assert f(torch.float32, False, 0, 10, 4) > 0
    for dtype in (torch.float32, torch.bfloat16):
        for grad in (False, True):
            assert f(dtype, grad, 64, 1000, 64) > 0
            # the pieces of the vocabulary bound it: four times the vocabulary, not four times the memory
            small, large = f(dtype, grad, 4096, 1 << 18, 1024), f(dtype, grad, 4096, 1 << 20, 1024)
            assert large < 2.5 * small and large < 4 << 30
    # forward and gradient keep no T x V array of the logits' size at the largest sizes
    assert f(torch.bfloat16, True, 8192, 1 << 20, 4096) < 8192 * (1 << 20)
    for bad in ((torch.float32, False, -1, 10, 4, 0), (torch.float32, False, 1, 0, 4, 0),
                (torch.float32, False, 1, 10, 0, 0), (torch.float32, False, 1, 10, 4, -1)):
        with pytest.raises(sg.SgemmArgumentError):
            f(*bad)


def test_errors_are_the_librarys():
    with pytest.raises(sg.SgemmArgumentError, match=r"vocab_ce: argument 6 \(X\) is invalid") as e:
        binding._raise(-6, "vocab_ce")
    assert e.value.code == -6 and isinstance(e.value, ValueError)
    with pytest.raises(sg.SgemmLaunchError, match="hipError_t 98"):
        binding._raise(98, "vocab_ce_grad")


def test_host_tensors_are_refused():
    X, W, t = torch.zeros(4, 8), torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensor"):
        sg.vocab_ce(X, W, t)
    with pytest.raises(TypeError):
        sg.vocab_ce([[1.0]], W, t)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sg.vocab_ce(X.double(), W, t)
    with pytest.raises(AttributeError):
        sg.vocab_nothing


# --- the tile loop's LDS layout ---------------------------------------------------------------
# A 128-bit read is served in four passes of 16 lanes, a 64-bit one in two of 32 lanes, over 64 banks.
PASSES_128 = [[l + 32 * h for l in (list(range(0, 4)) + list(range(12, 16)) + list(range(20, 28)))] for h in (0, 1)]
PASSES_128 += [[l + 32 * h for l in range(32) if l + 32 * h not in PASSES_128[h]] for h in (0, 1)]
PASSES_64 = [list(range(32)), list(range(32, 64))]


def conflict_free(addresses, size, passes):
    for lanes in passes:
        banks = [(addresses[l] + 4 * i) // 4 % 64 for l in lanes for i in range(size // 4)]
        if len(set(banks)) != len(banks):
            return False
    return True


def swz(r, u):
    return u ^ ((r >> 1) & 7)


def test_row_fragments_are_conflict_free():
    for r in range(64):
        assert sorted(swz(r, u) for u in range(8)) == list(range(8))
        assert all(swz(r, swz(r, u)) == u for u in range(8))
    for q in range(4):
        at = [(l & 31) * 128 + swz(l & 31, 2 * q + (l >> 5)) * 16 for l in range(64)]
        assert conflict_free(at, 16, PASSES_128)


@pytest.mark.parametrize("rows,planes", [(256, 1), (128, 1), (64, 1), (256, 2), (128, 2), (64, 2)])
def test_transposed_fragments_are_conflict_free(rows, planes):
    chunks = rows * planes // 32
    flip = (lambda r: r & 3) if chunks % 4 == 0 else (lambda r: (r >> 1) & 1)
    row = chunks * 64
    for c in range(chunks):
        for k0 in (0, 4, 16, 20):
            at = []
            for lane in range(64):
                i = lane & 15
                r = k0 + 8 * (lane >> 5) + (i >> 2)
                assert flip(r) == flip(i >> 2)  # a lane's flip does not depend on the step
                at.append(r * row + (c ^ flip(r)) * 64 + ((lane >> 4) & 1) * 32 + (i & 3) * 8)
            assert conflict_free(at, 8, PASSES_64)
    # every quad of a row is loaded from one place
    for r in range(8):
        assert sorted(u ^ (flip(r) << 2) for u in range(chunks * 4)) == list(range(chunks * 4))
