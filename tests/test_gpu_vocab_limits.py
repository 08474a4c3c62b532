"""GPU checks of the vocabulary head at the largest sizes that its calls take."""
import math

import pytest
import torch

import fp32_gemm_05_amd as sg

pytestmark = pytest.mark.gpu
LARGEST_VOCABULARY = 2 ** 31 - 1025


def test_largest_vocabulary_fp32_gradient():
    # W is 0 but for some rows, the last one among them: logits 0 and 1.  Its largest value, in the last row, is
    # past what an fp16 holds as it is, so it must have been found.
    V, T = LARGEST_VOCABULARY, 65
    W = torch.zeros(V, 1, device="cuda")
    rows = torch.tensor([V - 1, V - 4097, 2 ** 30 + 1, 0], device="cuda")
    W[rows] = 1e6
    X = torch.ones(T, 1, device="cuda")
    target = rows[torch.arange(T, device="cuda") % 4].clone()
    target[4] = V - 2  # a row of zeros
    lse = torch.full((T,), math.log(V + 4 * (math.e - 1)), device="cuda")
    dloss = torch.linspace(1, 2, T, device="cuda")
    dX, dW = sg.vocab_ce_grad(X, W, target, lse, dloss, alpha=1e-6, want_dw=False)
    assert dW is None
    # sum_v p W = 4 e / V: 5e-9 of W; lse and exp are off by a few 2^-24 of 21
    want = torch.where(torch.arange(T, device="cuda") == 4, 0.0, -dloss.double())[:, None]
    assert bool(((dX.double() - want).abs() <= 1e-5).all()), float((dX.double() - want).abs().max())
