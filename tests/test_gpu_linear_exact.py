"""GPU checks of the linear layer to the last bit, on every path: few tokens and many, products cut along their long axis
and not, operands read in place and packed (linear_exact.py)."""
import pytest
import torch

import fp32_gemm_05_amd as sg
import linear_exact as e
from linear_reference import ACTS, DT
from test_gpu_linear_range import slope

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 300, 4100), (7, 1000, 129), (16, 512, 256), (16, 40, 4000), (17, 65, 1000), (25, 8200, 60), (32, 1100, 3001),
         (33, 4097, 40), (40, 12300, 70), (48, 300, 2000), (57, 6200, 2100), (64, 130, 520), (64, 1500, 4096), (65, 64, 64),
         (66, 1, 7), (100, 257, 96), (130, 1000, 31), (257, 2049, 136), (515, 700, 1), (1000, 72, 2000), (2000, 1500, 777),
         (1030, 2056, 1032), (300, 100, 9000), (8191, 65, 33), (70, 20001, 64), (2048, 2304, 520), (4100, 4104, 72)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,H", SIZES)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_every_bit(T, N, H, dtype, pad):
    p = e.inputs(T, N, H, DT[dtype], "cuda", pad)
    for name in ("none", "relu"):
        Y, Z = sg.linear_act(p["X"], p["W"], p["bias"], p["residual"], activation=name, keep=True)
        y, z = e.forward(p, name)
        e.equal(Y, y, "Y")
        e.equal(Z, z, "Z")
    if dtype == "bf16":
        y, _ = e.forward(p, "relu", residual=False)
        e.equal(sg.linear_act(p["X"], p["W"], p["bias"], activation="relu", out_dtype=torch.float32), y, "wide Y")
    for name in ACTS:
        got = sg.linear_act_grad(p["X"], p["W"], p["dY"], p["Z"], activation=name)
        for g, w, what in zip(got, e.gradients(p, name), ("dX", "dW", "dbias")):
            e.equal(g, w, (name, what))
    alone = sg.linear_act_grad(p["X"], p["W"], p["dY"], p["Z"], activation="silu", want_dx=False, want_dw=False)[2]
    e.equal(alone, e.gradients(p, "silu")[2], "dbias alone")


@pytest.mark.parametrize("T", [9, 39, 63, 66, 999])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_dbias_is_summed_before_dz_is_rounded(T, name):
    """bf16: upstream gradients 3, -1, -2 in turn on one slope cancel to 0, off by a product's and T additions' 2^-24 of the terms'
    magnitudes each, and a last rounding.  Rounded to bf16 first, three terms would leave up to 2^-8 of themselves each time."""
    g = torch.Generator(device="cuda").manual_seed(T)
    N, bf16 = 200, torch.bfloat16
    X, W = torch.ones(T, 8, device="cuda", dtype=bf16), torch.ones(N, 8, device="cuda", dtype=bf16)
    dY = torch.tensor([3.0, -1.0, -2.0], device="cuda").repeat(T // 3)[:, None].expand(T, N).to(bf16).contiguous()
    Z = torch.randn(1, N, generator=g, device="cuda").to(bf16).expand(T, N).contiguous()
    one = slope(Z[0].double(), name)
    tol = (T + 2) * 2.0 ** -24 * T * 2 * one.abs() * (1 + 2.0 ** -8)
    dbias = sg.linear_act_grad(X, W, dY, Z, activation=name)[2].double()
    assert bool((dbias.abs() <= tol).all())
    lost = sum((k * one).to(bf16).double() for k in (3, -1, -2)) * (T // 3)
    assert float((lost.abs() > tol).double().mean()) > 0.5  # such a mistake would show
