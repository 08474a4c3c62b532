"""CPU checks of the vocabulary head's binding: what does not fit the C ABI's integers, streams of
other devices."""
import types

import pytest
import torch

import fp32_gemm_05_amd as sg
from fp32_gemm_05_amd import vocab as binding


@pytest.fixture
def any_device(monkeypatch):
    monkeypatch.setattr(binding, "_require_device", lambda t, name: None)


@pytest.mark.parametrize("shape,strides", [((3, 8), (2 ** 32 + 8, 1)), ((3, 8), (2 ** 31, 1)), ((2 ** 32 + 5, 1), (1, 1)),
                                           ((1, 2 ** 32 + 8), (2 ** 32 + 8, 1))])
def test_sizes_and_strides_past_32_bits_are_refused(any_device, shape, strides):
    for dtype in (torch.float32, torch.bfloat16):
        with pytest.raises(ValueError, match="above 2147483647"):
            binding._matrix(torch.empty_strided(shape, strides, dtype=dtype, device="meta"), "X")
    t = torch.empty_strided((3, 8), (2 ** 31 - 1, 1), device="meta")
    assert binding._matrix(t, "X") == (3, 8, 2 ** 31 - 1)
    # no stride is addressed in a single row
    assert binding._matrix(torch.empty_strided((1, 8), (2 ** 40, 1), device="meta"), "X") == (1, 8, 8)


@pytest.mark.parametrize("sizes,argument", [((2 ** 32 + 5, 10, 4, 0), 3), ((5, 2 ** 32 + 10, 4, 0), 4),
                                            ((5, 10, 2 ** 32 + 4, 0), 5), ((5, 10, 4, 2 ** 32), 6),
                                            ((2 - 2 ** 32, 10, 4, 0), 3)])
def test_workspace_of_sizes_past_32_bits_is_refused(sizes, argument):
    with pytest.raises(sg.SgemmArgumentError) as e:
        binding.vocab_workspace(torch.float32, True, *sizes)
    assert e.value.code == -argument


def test_ignored_target_past_64_bits_is_refused():
    assert binding._ignored(-2 ** 63) == -2 ** 63 and binding._ignored(True) == 1
    for index in (2 ** 63, 2 ** 64 - 100, -2 ** 63 - 1):
        with pytest.raises(ValueError, match="no int64"):
            binding._ignored(index)


def test_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    assert binding._on_device(stream, torch.device("cuda", 1)) is stream
    with pytest.raises(ValueError, match="stream is on cuda:1, X on cuda:0"):
        binding._on_device(stream, torch.device("cuda", 0))


def test_stream_of_another_device_is_refused_by_a_call(any_device, monkeypatch):
    entered = []
    monkeypatch.setattr(torch.cuda, "stream", entered.append)
    X = torch.empty(3, 8, device="meta")
    with pytest.raises(ValueError, match="stream is on cuda:1, X on meta"):
        binding._Problem(X, torch.empty(5, 8, device="meta"), 1.0, types.SimpleNamespace(device=torch.device("cuda", 1)))
    assert not entered
