"""GPU checks of the vocabulary head that a lost digit or a NaN does not pass: every path and tile shape against
float64, with the plain float32 form's own error as the measure (vocab_checks.check_digits)."""
import pytest
import torch

import fp32_gemm_05_amd as sg
import vocab_checks as vc

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# 1 to 64 tokens in each of their forms; above, shapes whose products take small, middle and large tiles, many
# slabs, rows read in place (whole slabs, and ends inside one) and packed; several pieces of the vocabulary
SIZES = [(1, 700, 320), (16, 9000, 321), (17, 3000, 200), (32, 20000, 130), (40, 3000, 777), (64, 13000, 512),
         (65, 1500, 600), (130, 777, 1000), (300, 1025, 64), (300, 20000, 1000), (500, 60000, 256), (1340, 3070, 174),
         (1000, 3001, 1000), (1362, 15116, 444), (2048, 32768, 512), (2142, 576, 3392), (1100, 140000, 136),
         (4100, 61000, 40)]


def inputs(T, V, H, dtype, spread, pad):
    g = torch.Generator(device="cuda").manual_seed(T + V)

    def rows(x):
        wide = torch.full((x.shape[0], H + pad), float("nan"), device="cuda", dtype=DT[dtype])
        wide[:, :H] = x
        return wide[:, :H]

    w = torch.randn(V, H, generator=g, device="cuda") * (spread / H ** 0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda") + 2 * torch.rand(T, 1, generator=g, device="cuda") * w[target]
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    return rows(x), rows(w), target, dloss, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", SIZES)
@pytest.mark.parametrize("spread", [1.5, 4.0])
def test_ce(T, V, H, dtype, spread):
    X, W, target, dloss, g = inputs(T, V, H, dtype, spread, 3 if spread == 4.0 else 0)
    if T > 1:
        target[::5] = -100
    index = torch.where(target >= 0, target, -1)[:, None]
    loss, lse = sg.vocab_ce(X, W, target)
    got = dict(zip(("dX", "dW"), sg.vocab_ce_grad(X, W, target, lse, dloss)), loss=loss, lse=lse)
    args = X, W, 1.0, index, torch.ones(T, 1, device="cuda"), target >= 0, dloss
    vc.check_digits(vc.definition(*args), vc.definition(*args, dtype=torch.float32), got, X.dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", SIZES)
@pytest.mark.parametrize("K", [3, 230])
def test_distill(T, V, H, dtype, K):
    X, W, _, dloss, g = inputs(T, V, H, dtype, 2.0, 8 if K == 3 else 0)
    index = torch.randint(0, V, (T, K), generator=g, device="cuda")
    index[torch.rand(T, K, generator=g, device="cuda") < 0.3] = -1
    if T > 1:
        index[::5] = -1
    teacher = torch.randn(T, K, generator=g, device="cuda")
    keep = index >= 0
    counts = keep.any(1)
    q = torch.softmax((teacher.double() * 0.8).masked_fill(~keep, -float("inf")), 1)
    q = torch.where(counts[:, None], q, 0.0)
    loss, lse, picked = sg.vocab_distill(X, W, index, teacher, alpha=0.5, teacher_alpha=0.8)
    got = dict(zip(("dX", "dW"), sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss, alpha=0.5,
                                                       teacher_alpha=0.8)), loss=loss, lse=lse)
    args = X, W, 0.5, index, q, counts, dloss
    vc.check_digits(vc.definition(*args), vc.definition(*args, dtype=torch.float32), got, X.dtype)
