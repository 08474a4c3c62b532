"""GPU checks of the vocabulary head's fp32 gradients where tokens differ in weight and magnitude.
Bounds: vocab_checks.py."""
import pytest
import torch

import fp32_gemm_05_amd as sg
import vocab_checks as vc

pytestmark = pytest.mark.gpu


def step(X, W, target, dloss, **kw):
    loss, lse = sg.vocab_ce(X, W, target, **kw)
    dX, dW = sg.vocab_ce_grad(X, W, target, lse, dloss, **kw)
    return {"loss": loss, "lse": lse, "dX": dX, "dW": dW}


def ce_definition(X, W, target, dloss, alpha=1.0):
    counts = target >= 0
    index = torch.where(counts, target, -1)[:, None]
    return vc.definition(X, W, alpha, index, torch.ones_like(index, dtype=torch.float64), counts, dloss)


def confident(T, V, H, margins, top, seed):
    """Tokens with a target logit of about `top` and one rival, the last row, `margin` below it, all else near 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda") * (0.05 / H ** 0.5)
    target = torch.randperm(V - 1, generator=g, device="cuda")[:T]
    # a common direction for the rival's row, a token's own for its target's
    common = torch.zeros(H, device="cuda")
    common[0] = 1.0
    x[:, 0] = 4.0
    margins = torch.tensor(margins, device="cuda")[torch.arange(T, device="cuda") % len(margins)]
    own = x.clone()
    own[:, 0] = 0.0
    W[target] = own * (top / own.square().sum(1, keepdim=True))
    W[V - 1] = common * ((top - 14.0) / 4.0)
    W[target] += common * ((margins - 14.0) / 4.0)[:, None]
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    return x, W, target, dloss


@pytest.mark.parametrize("T,V,H", [(100, 3000, 256), (300, 5003, 200), (900, 20000, 300)])
@pytest.mark.parametrize("counted", [1, 2, 4, "all"])
@pytest.mark.parametrize("top", [9.0, 25.0, 40.0])
def test_confident_tokens(T, V, H, counted, top):
    # 1 - p of the target from 1e-5 to below what fp32 can tell of z - lse
    X, W, target, dloss = confident(T, V, H, [15.0, 14.0, 16.0, 13.0, 18.0, 12.0], top, 3 + T)
    if counted != "all":
        target[torch.arange(T, device="cuda") >= counted] = -100
    got = step(X, W, target, dloss)
    for name in got:
        assert bool(torch.isfinite(got[name]).all()), name
    r = ce_definition(X, W, target, dloss)
    vc.check_fp32_gradients(r, got)
    # the rival's row takes p alone, whatever 1 - p of the targets is taken for
    v = V - 1
    a = (r["s"] * r["p"])[:, v:v + 1].t().abs()
    bound = (a * (r["E"] + (4 * T ** 0.5 + 8) * vc.U)) @ X.double().abs()
    vc.rows_within("rival", got["dW"][v:v + 1], r["dW"][v:v + 1], bound)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,H", [(40, 3000, 256), (100, 3000, 256), (900, 20000, 300)])
@pytest.mark.parametrize("top", [25.0, 40.0])
def test_cross_entropy_is_not_negative(T, V, H, top, dtype):
    X, W, target, dloss = confident(T, V, H, [12.0, 14.0, 16.0, 18.0, 20.0], top, 5 + T)
    X, W = X.to(dtype), W.to(dtype)
    loss, _ = sg.vocab_ce(X, W, target)
    r = ce_definition(X, W, target, dloss)
    assert bool((loss >= 0).all()), float(loss.min())
    # lse and z are off by E / 4 each at most but for one in 10^4, and their difference by what both are
    assert bool(((loss.double() - r["loss"]).abs() <= r["E"]).all())
    target[::2] = V  # outside the vocabulary: still NaN
    assert bool(torch.isnan(sg.vocab_ce(X, W, target)[0][::2]).all())


@pytest.mark.parametrize("T,V,H", [(100, 1500, 96), (300, 20000, 200)])
@pytest.mark.parametrize("alpha", [1e5, -1e6, 1e7])
def test_logits_beyond_what_fp32_tells_apart(T, V, H, alpha):
    # z - lse may be off by 1 and more: p is then any value up to 1, and nothing overflows
    g = torch.Generator(device="cuda").manual_seed(T)
    X = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda") * (1.5 / H ** 0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    index = torch.randint(0, V, (T, 3), generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    got = step(X, W, target, dloss, alpha=alpha)
    loss, lse, picked = sg.vocab_distill(X, W, index, torch.zeros(T, 3, device="cuda"), alpha=alpha)
    got["dX of distillation"], got["dW of distillation"] = sg.vocab_distill_grad(
        X, W, index, torch.zeros(T, 3, device="cuda"), lse, picked, dloss, alpha=alpha)
    for name in got:
        assert bool(torch.isfinite(got[name]).all()), name


PATHS = [(5, 700, 96), (40, 700, 96), (150, 1500, 96), (900, 20000, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", PATHS)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_one_tokens_upstream_gradient_stays_its_own(T, V, H, dtype, value):
    g = torch.Generator(device="cuda").manual_seed(T)
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    X = torch.randn(T, H, generator=g, device="cuda").to(t)
    W = (torch.randn(V, H, generator=g, device="cuda") * (1.5 / H ** 0.5)).to(t)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    index = torch.randint(0, V, (T, 3), generator=g, device="cuda")
    teacher = torch.randn(T, 3, generator=g, device="cuda")
    bad = T // 2
    others = torch.arange(T, device="cuda") != bad
    dloss[bad] = value
    loss, lse = sg.vocab_ce(X, W, target)
    ce = sg.vocab_ce_grad(X, W, target, lse, dloss)[0]
    _, lse, picked = sg.vocab_distill(X, W, index, teacher)
    distill = sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss)[0]
    dloss[bad] = 1.0
    _, lse_ce = sg.vocab_ce(X, W, target)
    clean = sg.vocab_ce_grad(X, W, target, lse_ce, dloss)[0], \
        sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss)[0]
    for got, want in zip((ce, distill), clean):
        assert bool(torch.isfinite(got[others]).all())
        assert not bool(torch.isfinite(got[bad]).all())
        # what the other tokens are rounded in may follow the largest weight
        vc.rows_within("dX", got[others], want[others], 2.0 ** -18 * want[others].double().abs())


@pytest.mark.parametrize("T,V,H", [(100, 1500, 96), (777, 5003, 200), (200, 32768, 256)])
@pytest.mark.parametrize("scale", [1.0, 1e-2, 1e-4])
@pytest.mark.parametrize("small", [0.0, 1e-9])
def test_a_row_of_zeros_among_others(T, V, H, scale, small):
    # a counted row of zeros, or a very small one, takes nothing from the other tokens, and its own dX is as exact
    g = torch.Generator(device="cuda").manual_seed(T + H)
    X = torch.randn(T, H, generator=g, device="cuda") * scale
    W = torch.randn(V, H, generator=g, device="cuda") * (1.5 / H ** 0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    X[T // 3] *= small
    vc.check_fp32_gradients(ce_definition(X, W, target, dloss), step(X, W, target, dloss))


@pytest.mark.parametrize("T,V,H", [(100, 1500, 96), (777, 5003, 200)])
def test_weights_far_apart(T, V, H):
    # a token's dX is as exact beside upstream gradients 10^6 times its own
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    X = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda") * (1.5 / H ** 0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    dloss[::3] *= 1e6
    dloss[1::3] *= -1e-3
    vc.check_fp32_gradients(ce_definition(X, W, target, dloss), step(X, W, target, dloss))


@pytest.mark.parametrize("T,V,H", PATHS)
@pytest.mark.parametrize("value", [float("inf"), 1e38, 1e-30])
def test_a_tokens_dx_does_not_depend_on_other_tokens(T, V, H, value):
    g = torch.Generator(device="cuda").manual_seed(T + 2)
    X = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda") * (1.5 / H ** 0.5)
    index = torch.randint(0, V, (T, 3), generator=g, device="cuda")
    teacher = torch.randn(T, 3, generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    bad = T // 2
    others = torch.arange(T, device="cuda") != bad
    got = []
    for change in (False, True):
        if change:
            dloss[bad] = value
            X[bad] *= 1e-6
        _, lse, picked = sg.vocab_distill(X, W, index, teacher)
        got.append(torch.stack([step(X, W, index[:, 0].contiguous(), dloss)["dX"][others],
                                sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss)[0][others]]))
    assert bool(torch.isfinite(got[0]).all()) and torch.equal(got[0], got[1])
