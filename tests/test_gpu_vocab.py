"""GPU checks of the vocabulary-head operators against a plain float64 implementation.

Tolerances (derived, not tuned).  u = 2^-24 is half a step of fp32, b = 2^-8 the largest relative
rounding error of bf16.

loss, lse, picked: a logit is a sum of H products, off by at most H * u * alpha * sum|x w| =: H u S
(fp32 operands in two fp16 planes add under 4 u a product: two roundings and the dropped low x low);
exp and log of values of magnitude m are off by a few (m + 2) u.  So |error| <= (H + 64) * u *
(S + |lse| + 2) + F, S the largest sum|x w| * alpha of the token's logits; a distillation loss adds
K terms of the same kind.  F is the two planes' floor: a value is held to 2^-40 of the largest of its
row of X (of its matrix, for W), so F = H * 2^-39 * alpha * max|x| * max|w|.

dX, dW: with D the exact d(loss)/dz, an element is a sum over n terms (n = V or T).  fp32: D's own
relative error is (H + 64) u (S + |lse| + 2) plus 2^-20 for its exp and products, the sum adds n u:
|error| <= (((H + 64)(S + |lse| + 2) + n + 64) u + F) * A, A = sum over |alpha dloss| (p + y) |w| (the
absolute terms), plus D's own floor: its entries are held to 2^-40 of max|alpha dloss x| / max|x| of
the token, so n * 2^-39 * max|alpha dloss x| for dW, times max|w| / max|x of the token| for dX.  bf16 adds b for D, b for the scaled X of cross entropy, and b |result| for the
final rounding: 3 b A in all.
"""
import pytest
import torch

import fp32_gemm_05_amd as sg

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(T, V, H, dtype, seed, pad=0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(x):
        wide = torch.full((x.shape[0], H + pad), float("nan"), device="cuda", dtype=DT[dtype])
        wide[:, :H] = x
        return wide[:, :H]

    w = torch.randn(V, H, generator=g, device="cuda") * (spread / H ** 0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda") + 2 * torch.rand(T, 1, generator=g, device="cuda") * w[target]
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    return rows(x), rows(w), target, dloss, g


def entries(T, V, K, g, none=0.3):
    index = torch.randint(0, V, (T, K), generator=g, device="cuda")
    index[torch.rand(T, K, generator=g, device="cuda") < none] = -1
    return index, torch.randn(T, K, generator=g, device="cuda")


def reference(X, W, alpha, index, q, counts, dloss):
    """float64: loss, lse, D, and the absolute terms, for targets given as entries with weights q."""
    x, w = X.double(), W.double()
    x = torch.where(counts[:, None], x, 0.0)
    z = alpha * (x @ w.t())
    S = abs(alpha) * (x.abs() @ w.abs().t()).max(1).values
    lse = torch.logsumexp(z, 1)
    keep = index >= 0
    at = index.clamp(min=0)
    y = torch.zeros_like(z).scatter_add_(1, at, q * keep)
    picked = torch.where(keep, z.gather(1, at), 0.0)
    loss = torch.where(keep & (q > 0), q * (q.clamp(min=1e-300).log() - picked + lse[:, None]), 0.0).sum(1)
    s = torch.where(counts, alpha * dloss.double(), 0.0)[:, None]
    p = (z - lse[:, None]).exp()
    T, H = X.shape
    most = (s.abs() * x.abs()).max()
    zero = lambda v: torch.where(counts, v, 0.0)  # noqa: E731
    return {"loss": zero(loss), "lse": zero(lse), "picked": torch.where(counts[:, None], picked, 0.0), "S": S,
            "dX": s * (p - y) @ w, "dW": (s * (p - y)).t() @ x,
            "F": H * 2.0 ** -39 * abs(alpha) * x.abs().amax(1) * w.abs().max(),
            "GW": T * 2.0 ** -39 * most,
            "GX": (W.shape[0] * 2.0 ** -39 * most * w.abs().max() / x.abs().amax(1).clamp(min=1e-30))[:, None],
            "AX": s.abs() * (p + y) @ w.abs(), "AW": (s.abs() * (p + y)).t() @ x.abs()}


def check(r, X, W, got, dtype, K):
    T, H, V = X.shape[0], X.shape[1], W.shape[0]
    head = (H + 64) * (r["S"] + r["lse"].abs() + 2) + r["F"] / U
    for name in ("loss", "lse"):
        err = (got[name].double() - r[name]).abs()
        assert bool((err <= (head + (K * (r["lse"].abs() + 8) if name == "loss" else 0)) * U).all()), \
            (name, float(err.max()))
    if "picked" in got:
        err = (got["picked"].double() - r["picked"]).abs()
        assert bool((err <= head[:, None] * U).all()), float(err.max())
    top = head.max() if T else 0.0
    for name, n, a in (("dX", V, "AX"), ("dW", T, "AW")):
        if got.get(name) is None:
            continue
        assert got[name].dtype == X.dtype
        tol = (top + n + 64) * U + (3 * B if dtype == "bf16" else 0)
        err = (got[name].double() - r[name]).abs()
        tol = tol * r[a] + r["G" + name[1]] + 1e-37
        bad = err > tol
        assert not bool(bad.any()), (name, int(bad.sum()), float((err / tol).max()))


def run_ce(X, W, target, dloss, alpha=1.0, dtype="f32", ignore=-100):
    counts = target != ignore
    idx = torch.where(counts, target, -1)[:, None]
    loss, lse = sg.vocab_ce(X, W, target, alpha=alpha, ignore_index=ignore)
    dX, dW = sg.vocab_ce_grad(X, W, target, lse, dloss, alpha=alpha, ignore_index=ignore)
    r = reference(X, W, alpha, idx, torch.ones_like(idx, dtype=torch.double), counts, dloss)
    check(r, X, W, {"loss": loss, "lse": lse, "dX": dX, "dW": dW}, dtype, 1)
    return loss, lse, dX, dW


def run_distill(X, W, index, teacher, dloss, alpha, teacher_alpha, dtype):
    keep = index >= 0
    counts = keep.any(1)
    t = (teacher.double() * teacher_alpha).masked_fill(~keep, -float("inf"))
    q = torch.where(counts[:, None], torch.softmax(t, 1), 0.0)
    loss, lse, picked = sg.vocab_distill(X, W, index, teacher, alpha=alpha, teacher_alpha=teacher_alpha)
    dX, dW = sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss, alpha=alpha, teacher_alpha=teacher_alpha)
    r = reference(X, W, alpha, index, q, counts, dloss)
    check(r, X, W, {"loss": loss, "lse": lse, "picked": picked, "dX": dX, "dW": dW}, dtype, index.shape[1])
    return loss, lse, picked, dX, dW


SIZES = [(1, 1, 1), (1, 500, 64), (3, 257, 33), (16, 1000, 128), (64, 512, 64), (65, 4097, 200), (130, 777, 65),
         (256, 2048, 256), (300, 5003, 129), (1000, 3001, 320), (129, 50000, 257), (2050, 6400, 512),
         # rows of whole slabs, read in place, and a vocabulary whose last 256 rows hold a whole empty tile
         (22, 1152, 192), (300, 1025, 64), (700, 33000, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", SIZES)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_ce(T, V, H, dtype, pad):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 11 + T, pad)
    run_ce(X, W, target, dloss, 1.0, dtype)
    target[torch.rand(T, generator=g, device="cuda") < 0.5] = -100
    run_ce(X, W, target, dloss, 0.7, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", SIZES)
@pytest.mark.parametrize("K", [1, 5, 70])
def test_distill(T, V, H, dtype, K):
    X, W, _, dloss, g = inputs(T, V, H, dtype, 23 + T, 3 if K == 5 else 0)
    index, teacher = entries(T, V, K, g)
    run_distill(X, W, index, teacher, dloss, 0.5, 0.8, dtype)
