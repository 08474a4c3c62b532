"""GPU checks of the linear layer over the whole range of its values: activations and their slopes far out, relative to
themselves, against 64 bits.

With one hidden element and a weight of 1, Z is X, Y the activation and dX of dY = 1 its slope, which passes the products
whole: exactly in fp32, as three bf16 parts to 2^-24, as two to 2^-16; one rounding of the result, u = 2^-24 or 2^-8.
"""
import math

import pytest
import torch

import fp32_gemm_05_amd as sg
from linear_reference import DT, rounded

pytestmark = pytest.mark.gpu
FAR = ("gelu", "gelu_tanh", "silu")


def slope(z, name):
    """act' in 64 bits, with all its digits on the far negative side."""
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a, b = 2 * math.sqrt(2 / math.pi), 0.044715
    w, rise = (z, torch.ones_like(z)) if name == "silu" else (a * (z + b * z ** 3), a * (1 + 3 * b * z * z))
    s = torch.special.expit(w)
    return s * (1 + z * rise * torch.special.expit(-w))


def own_error(z, name):
    """What a slope may be off by, of itself, where it is not near its zero: 2^-19 for exponential, reciprocal, tail and
    the products around them, and what the exponent is off by.  It is a product of fp32 roundings, each 2^-24 of it: z / 2
    times a constant, twice, for silu; w of five roundings and a constant for gelu_tanh; of gelu it is held in two parts."""
    exponent = {"silu": z.abs() * 2, "gelu": torch.zeros_like(z), "gelu_tanh": 7 * 1.6 * (z.abs() + 0.0448 * z.abs() ** 3)}[name]
    return 2.0 ** -19 + 2.0 ** -24 * exponent


def points(dtype):
    z = torch.cat([torch.tensor([-21.0, -25.0, -30.0, -60.0, -80.0, -86.0, -88.5, -95.0, -103.0, -110.0, -1e4, -1e30, 20.0, 25.0, 1e30]),
                   torch.linspace(-100, -2, 1171), torch.linspace(1, 22, 37)])
    return z.to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", FAR)
@pytest.mark.parametrize("T", [5, 16, 30, 64, 500])
def test_slopes_far_out(name, dtype, T):
    one = torch.ones(1, 1, device="cuda", dtype=DT[dtype])
    for z in points(dtype).split(T):
        z = z[:, None].contiguous()
        dY = torch.ones_like(z)
        dX, dW, dbias = sg.linear_act_grad(z, one, dY, z, activation=name)
        want = slope(z.double(), name)
        # below the smallest normal number digits are lost, those of the parts that a product takes too
        floor = 2.0 ** -125
        parts = 2.0 ** -16 if dtype == "bf16" and z.shape[0] <= 64 else rounded(dX, dX.dtype)
        tol = want.abs() * (own_error(z.double(), name) + parts + rounded(dX, dX.dtype)) + floor
        bad = ~((dX.double() - want).abs() <= tol)
        assert not bool(bad.any()), (z[bad].tolist()[:5], dX[bad].tolist()[:5], want[bad].tolist()[:5])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_unit_that_is_off_gets_nothing(dtype):
    """dW, dbias and dX of units whose Z is far below 0 for all tokens."""
    for T in (20, 300):
        X, W = torch.ones(T, 64, device="cuda", dtype=DT[dtype]), torch.ones(40, 64, device="cuda", dtype=DT[dtype])
        dY, Z = torch.ones(T, 40, device="cuda", dtype=DT[dtype]), torch.full((T, 40), -200.0, device="cuda", dtype=DT[dtype])
        for name in FAR:
            for g in sg.linear_act_grad(X, W, dY, Z, activation=name):
                assert not g.any(), (name, T)


@pytest.mark.parametrize("T", [5, 30, 500])
def test_far_side_of_gelu(T):
    """gelu(z) = z Phi(z) of negative z, relative to itself.

    The tail's polynomial is off by 2.3e-7; in steps u = 2^-24 of fp32, its steps by 2 u (each adds less than 0.6 of the one
    before), its argument by 3 u (a reciprocal and its sum) times 1.7, how steep it is, the exponential's square by 2 (2 u + u),
    its last place and the low part's factor, and three products by u each: 16 u + 2.3e-7 < 1.2e-6 < 2^-19."""
    z = torch.linspace(-13, -1, 3000).cuda()
    one = torch.ones(1, 1, device="cuda")
    for x in z.split(T):
        Y = sg.linear_act(x[:, None].contiguous(), one, activation="gelu")[:, 0]
        x = x.double()
        want = x * 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
        bad = ~((Y.double() - want).abs() <= 2.0 ** -19 * want.abs() + 2.0 ** -126)
        assert not bool(bad.any()), (x[bad].tolist()[:5], Y[bad].tolist()[:5], want[bad].tolist()[:5])


def same(got, want):
    """Infinities and NaN where 64 bits have them."""
    assert bool((got.isnan() == want.isnan()).all()) and bool((got.isinf() == want.isinf()).all())
    assert bool((got.sign() == want.sign())[got.isinf()].all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,H", [(16, 70, 100), (17, 70, 100), (20, 9000, 70), (32, 300, 2051), (37, 77, 1000), (50, 130, 33),
                                   (64, 12300, 64), (64, 6200, 2100), (65, 70, 100)])
def test_infinities_whatever_the_number_of_tokens(dtype, T, N, H):
    """In X, in W, and both signs in one sum; the other rows' and columns' bits stay as they are."""
    g = torch.Generator(device="cuda").manual_seed(T)
    X = torch.randn(T, H, generator=g, device="cuda").to(DT[dtype])
    W = torch.randn(N, H, generator=g, device="cuda").to(DT[dtype])
    clean = sg.linear_act(X, W)
    for value in (math.inf, -math.inf, math.nan):
        for t, n, h in ((T - 1, N - 1, H - 1), (0, 0, 0), (T // 2, N // 2, H // 2)):
            x = X.clone()
            x[t, h] = value
            y = sg.linear_act(x, W)
            same(y, x.double() @ W.double().t())
            y[t] = clean[t]
            assert torch.equal(y, clean)
            w = W.clone()
            w[n, h] = value
            y = sg.linear_act(X, w)
            same(y, X.double() @ w.double().t())
            y[:, n] = clean[:, n]
            assert torch.equal(y, clean)
    x, w = X.clone(), W.clone()
    x[1, 0], x[1, H - 1], w[2, 1] = math.inf, -math.inf, -math.inf
    x[3, 1] = 0.0  # times an infinity
    same(sg.linear_act(x, w), x.double() @ w.double().t())
    x = X.clone()
    x[T - 1] = -math.inf
    w = W.abs() + 1
    y = sg.linear_act(x, w, activation="relu")
    assert not y[T - 1].any() and bool(y.isfinite().all())


@pytest.mark.parametrize("T", [5, 20, 37, 50, 64, 100])
@pytest.mark.parametrize("name", ["none", "relu"])
def test_largest_numbers(T, name):
    """fp32 values up to the largest: sums of one such product and others of its scale, within an fp32 sum's error."""
    g = torch.Generator(device="cuda").manual_seed(T)
    most, N, H = torch.finfo(torch.float32).max, 90, 77
    X = torch.randn(T, H, generator=g, device="cuda") * 1e30
    X[:, 5] = most * (1 - 2.0 ** -12 * torch.rand(T, generator=g, device="cuda"))
    X[::3, 5] = -most
    W = torch.randn(N, H, generator=g, device="cuda")
    W[:, 5] = 0.25 + 0.5 * torch.rand(N, generator=g, device="cuda")
    Y = sg.linear_act(X, W, activation=name)
    x, w = X.double(), W.double()
    want, S = x @ w.t(), x.abs() @ w.abs().t()
    want = want.clamp(min=0) if name == "relu" else want
    assert bool(((Y.double() - want).abs() <= (H + 8) * 2.0 ** -24 * S).all())


def test_far_out_whatever_the_number_of_tokens():
    """Activations at the ends of the range."""
    z = torch.tensor([-3e38, -1e20, -1e4, -60.0, 21.0, 60.0, 1e4, 1e20, 3e38, math.inf, math.nan], device="cuda")
    n, W = len(z), torch.ones(1, 1, device="cuda")
    for times in (1, 2, 4, 5, 10):
        x = z.repeat(times)[:, None].contiguous()
        for name in ("relu", "gelu", "gelu_tanh", "silu"):
            Y, Z = sg.linear_act(x, W, activation=name, keep=True)
            assert torch.equal(Z[:n - 1], x[:n - 1]) and bool(Z[n - 1].isnan())
            assert torch.equal(Y[4:n - 1], x[4:n - 1]) and bool(Y[n - 1].isnan())
            # z exp(z) at -60: 5e-25
            assert bool((Y[:4].abs() < 1e-24).all())
