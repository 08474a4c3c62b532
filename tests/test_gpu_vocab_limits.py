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


# one wave for four entries would be more than 2^32 threads
@pytest.mark.parametrize("T,K", [(4096, 2 ** 16 + 60), (64, 2 ** 22 + 60)])
def test_entries_past_a_grids_threads(T, K):
    V, H = 300, 16
    assert T * (K // 4) * 64 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(T)
    X = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda") / 4
    few = torch.randint(0, V, (T, 2), generator=g, device="cuda")
    few_teacher = torch.randn(T, 2, generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    index = torch.full((T, K), -1, device="cuda")
    teacher = torch.full((T, K), float("nan"), device="cuda")
    index[:, 0], index[:, -1] = few[:, 0], few[:, 1]
    teacher[:, 0], teacher[:, -1] = few_teacher[:, 0], few_teacher[:, 1]
    want = sg.vocab_distill(X, W, few, few_teacher)
    got = sg.vocab_distill(X, W, index, teacher)
    # the same two entries, in the same order
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[2][:, 0], want[2][:, 0]) and torch.equal(got[2][:, -1], want[2][:, 1])
    assert not bool(got[2][:, 1:-1].any())
    want = sg.vocab_distill_grad(X, W, few, few_teacher, *want[1:], dloss)
    got = sg.vocab_distill_grad(X, W, index, teacher, *got[1:], dloss)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [64, 1000])
def test_no_tokens_to_distill(dtype, H):
    # the gradient of nothing: dW is set to 0, in the workspace that the call asked for
    from fp32_gemm_05_amd import vocab as binding
    V, K = 700, 5
    W = torch.randn(V, H, device="cuda").to(dtype)
    n = sg.vocab_workspace(dtype, True, 0, V, H, K)
    memory = torch.full((n + 2 ** 20,), 77, dtype=torch.uint8, device="cuda")
    dW = torch.full((V, H), float("nan"), device="cuda", dtype=dtype)
    binding._Problem(torch.empty(0, H, device="cuda", dtype=dtype), W, 1.0, None, K).call(
        "vocab_distill_grad", memory[:n], binding._TYPES[dtype], 0, V, H, K, 1.0, 1.0, None, H, W.data_ptr(), H, None, K,
        None, K, None, None, None, None, H, dW.data_ptr(), H)
    torch.cuda.synchronize()
    assert not bool(dW.any()) and bool((memory[n:] == 77).all())
    none = torch.empty(0, K, dtype=torch.int64, device="cuda")
    X = torch.empty(0, H, device="cuda", dtype=dtype)
    loss, lse, picked = sg.vocab_distill(X, W, none, none.float())
    dX, dW = sg.vocab_distill_grad(X, W, none, none.float(), lse, picked, loss)
    assert loss.shape == lse.shape == (0,) and picked.shape == (0, K) and dX.shape == (0, H) and not bool(dW.any())
