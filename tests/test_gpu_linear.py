"""GPU checks of the linear layer with an epilogue against a plain implementation in 64 bits
(linear_reference.py, which derives the tolerances)."""
import pytest
import torch

import fp32_gemm_05_amd as sg
from linear_reference import ACTS, DT, check_forward, check_gradients

pytestmark = pytest.mark.gpu


def padded(x, pad, fill=float("nan")):
    wide = torch.full((x.shape[0], x.shape[1] + pad), fill, device="cuda", dtype=x.dtype)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def inputs(T, N, H, dtype, pad=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T * 7 + N)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    X = padded(rand(T, H).to(DT[dtype]), pad)
    W = padded((rand(N, H) / H ** 0.5 * 1.5).to(DT[dtype]), pad)
    return X, W, rand(N).to(DT[dtype]), padded(rand(T, N).to(DT[dtype]), pad), padded(rand(T, N).to(DT[dtype]), pad)


def step(T, N, H, dtype, name, pad=0, bias=True, residual=True):
    X, W, b, R, dY = inputs(T, N, H, dtype, pad)
    b, R = b if bias else None, R if residual else None
    keep = name != "none"
    out = sg.linear_act(X, W, b, R, activation=name, keep=keep)
    Y, Z = out if keep else (out, None)
    check_forward(X, W, b, R, name, Y, Z)
    dX, dW, dbias = sg.linear_act_grad(X, W, dY, Z, activation=name)
    check_gradients(X, W, b, dY, name, dX, dW, dbias)


SIZES = [(1, 1, 1), (1, 64, 64), (2, 300, 33), (7, 1000, 129), (16, 512, 256), (17, 65, 1000), (33, 4097, 40),
         (64, 130, 520), (65, 64, 64), (66, 1, 7), (100, 257, 96), (128, 128, 1000), (130, 1000, 31), (300, 513, 520),
         (257, 2049, 136), (1000, 72, 2000), (515, 700, 1), (2000, 1500, 777), (1030, 2056, 1032)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,H", SIZES)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_sizes(T, N, H, dtype, pad):
    step(T, N, H, dtype, "gelu" if pad else "none", pad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,H", [(33, 12300, 70), (40, 12290, 1000), (48, 300, 2000), (37, 500, 4001), (44, 6200, 2100),
                                   (49, 300, 1500), (53, 3003, 3000), (64, 1500, 4096), (33, 5504, 1100), (20, 70, 2000), (32, 1100, 3001), (5, 40, 4000), (16, 1000, 2050)])
def test_few_tokens(T, N, H, dtype):
    """Numbers of tokens between those that fill the matrix instructions, long sums of few output features."""
    step(T, N, H, dtype, "silu", 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T,N,H", [(3, 200, 100), (40, 256, 64), (200, 384, 256)])
@pytest.mark.parametrize("bias,residual", [(True, False), (False, True), (False, False), (True, True)])
def test_epilogues(T, N, H, dtype, name, bias, residual):
    step(T, N, H, dtype, name, 0, bias, residual)
