"""CPU checks that the bounds of vocab_checks.py see what they are there for: the fp32 operators' arithmetic
(operands in two fp16 planes, three products) is emulated and passes, and with a mistake planted in it does not."""
import pytest
import torch

import vocab_checks as vc

T, V, H = 130, 900, 320


def planes(x, unit_of, keep=None):
    """x as the sum of two fp16 values after scaling by a power of two; `keep`: a mask of where the low one stays."""
    top = x.abs().amax(unit_of, keepdim=True) if unit_of is not None else x.abs().max()
    scale = torch.exp2(14 - torch.floor(torch.log2(torch.where(top > 0, top, 1.0))))
    y = x * scale
    high = y.half().float()
    low = (y - high).half().float()
    if keep is not None:
        low = torch.where(keep, low, 0.0)
    return high / scale, low / scale


def product(a, b):
    """a b^T of planes, without low times low."""
    return a[0] @ b[1].t() + a[1] @ b[0].t() + a[0] @ b[0].t()


def emulated(X, W, target, dloss, mistake=None):
    counts = target >= 0
    s = torch.where(counts, dloss, 0.0)[:, None]
    slabs = torch.arange(H) < 96  # three slabs
    px = planes(X, 1, {"x low": torch.zeros(H, dtype=torch.bool), "x low past slabs": slabs}.get(mistake))
    pw = planes(W, 1, torch.zeros(H, dtype=torch.bool) if mistake == "w low" else None)
    z = product(px, pw)
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(counts, lse - zt, 0.0)
    d = (z - lse[:, None]).exp()
    d[torch.arange(T), target.clamp(min=0)] -= 1
    d = torch.where(counts[:, None], d, 0.0)
    no = torch.zeros(1, dtype=torch.bool)
    one = torch.full((T, 1), 1.0)  # D's scale is that of 1
    pd = [v[:, 1:] for v in planes(torch.cat([one, d], 1), 1, no if mistake == "d low" else None)]
    if mistake == "d row":
        pd[0][7] = pd[0][6]
    px = planes(X * s, None, no if mistake == "s x low" else None)
    pw = planes(W, None)
    dX = s * product(pd, [v.t() for v in pw])
    dW = product([v.t() for v in pd], [v.t() for v in px])
    if mistake == "nan":
        dW[3, 5] = float("nan")
    if mistake == "dx part":  # a part of the vocabulary left out
        dX -= s * (d[:, -3:] @ W[-3:])
    return {"loss": loss, "lse": torch.where(counts, lse, 0.0), "dX": dX, "dW": dW}


def case(spread, seed):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(V, H, generator=g) * (spread / H ** 0.5)
    target = torch.randint(0, V, (T,), generator=g)
    X = torch.randn(T, H, generator=g) + 2 * torch.rand(T, 1, generator=g) * W[target]
    dloss = torch.rand(T, generator=g) + 0.5
    target[::5] = -100
    index = torch.where(target >= 0, target, -1)[:, None]
    args = X, W, 1.0, index, torch.ones(T, 1), target >= 0, dloss
    return (X, W, target, dloss), vc.definition(*args), vc.definition(*args, dtype=torch.float32)


@pytest.mark.parametrize("spread", [1.5, 4.0])
def test_the_arithmetic_passes(spread):
    inputs, r, plain = case(spread, 1)
    got = emulated(*inputs)
    vc.check_fp32_gradients(r, got)
    vc.check_digits(r, plain, got, torch.float32)
    vc.check_digits(r, plain, plain, torch.float32)


@pytest.mark.parametrize("mistake", ["x low", "x low past slabs", "w low", "d low", "s x low", "d row", "nan", "dx part"])
def test_a_mistake_is_seen(mistake):
    inputs, r, plain = case(4.0, 2)
    with pytest.raises(AssertionError):
        vc.check_digits(r, plain, emulated(*inputs, mistake), torch.float32)


@pytest.mark.parametrize("mistake", ["d row", "nan"])
def test_a_mistake_is_seen_by_the_gradients_bound(mistake):
    inputs, r, _ = case(1.5, 3)
    with pytest.raises(AssertionError):
        vc.check_fp32_gradients(r, emulated(*inputs, mistake))
