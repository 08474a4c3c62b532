"""GPU checks of the vocabulary-head operators where they can go wrong: tokens that do not count and what
their rows hold, targets outside the vocabulary, streams, graphs, pieces, long strides, differences.
The plain implementation and the tolerances are those of test_gpu_vocab.py."""
import importlib.util
import os

import pytest
import torch

import fp32_gemm_05_amd as sg
from test_gpu_vocab import DT, check, entries, inputs, reference, run_ce, run_distill

pytestmark = pytest.mark.gpu
# both paths: at most 64 tokens, and more (small and large tiles)
PATHS = [(5, 700, 96), (40, 700, 96), (150, 1500, 96), (900, 20000, 128)]


def step(X, W, target, dloss, **kw):
    loss, lse = sg.vocab_ce(X, W, target, **kw)
    return (loss, lse) + sg.vocab_ce_grad(X, W, target, lse, dloss, **kw)


def distill_step(X, W, index, teacher, dloss, **kw):
    loss, lse, picked = sg.vocab_distill(X, W, index, teacher, **kw)
    return (loss, lse, picked) + sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss, **kw)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", PATHS)
def test_rows_that_do_not_count_reach_nothing(T, V, H, dtype):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 5)
    index, teacher = entries(T, V, 4, g)
    out = torch.rand(T, generator=g, device="cuda") < 0.4
    out[0] = True
    target[out] = -100
    index[out] = -1
    clean = step(X, W, target, dloss), distill_step(X, W, index, teacher, dloss)
    X, dloss, teacher = X.clone(), dloss.clone(), teacher.clone()
    X[out], dloss[out], teacher[out] = float("nan"), float("inf"), float("nan")
    teacher[index < 0] = float("inf")
    dirty = step(X, W, target, dloss), distill_step(X, W, index, teacher, dloss)
    for a, b in zip(clean, dirty):
        assert same(a, b)
        assert all(bool(torch.isfinite(x).all()) for x in b)
        assert not bool(b[0][out].any()) and not bool(b[1][out].any()) and not bool(b[-2][out].any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 33, 100, 700])
def test_no_token_counts(T, dtype):
    X, W, target, dloss, g = inputs(T, 900, 80, dtype, 6)
    index, teacher = entries(T, 900, 3, g, none=2.0)
    for got in (step(X, W, torch.full_like(target, -100), dloss), distill_step(X, W, index, teacher, dloss)):
        assert all(not bool(x.any()) for x in got)
        assert got[-2].shape == X.shape and got[-1].shape == W.shape


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens(dtype):
    X, W, target, dloss, _ = inputs(3, 500, 64, dtype, 7)
    loss, lse, dX, dW = step(X[:0], W, target[:0], dloss[:0])
    assert loss.shape == lse.shape == (0,) and dX.shape == (0, 64)
    assert dW.shape == (500, 64) and not bool(dW.any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", PATHS)
@pytest.mark.parametrize("wrong", [-1, 10 ** 12, "V"])
def test_target_outside_the_vocabulary_is_nan(T, V, H, dtype, wrong):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 8)
    before = step(X, W, target, dloss)
    bad = T // 2
    target[bad] = V if wrong == "V" else wrong
    loss, lse, dX, dW = step(X, W, target, dloss)
    others = torch.arange(T, device="cuda") != bad
    assert bool(torch.isnan(loss[bad])) and bool(torch.isnan(dX[bad]).all()) and bool(torch.isnan(dW).all())
    assert torch.equal(loss[others], before[0][others]) and torch.equal(lse, before[1])
    assert bool(torch.isfinite(dX[others]).all())
    index, teacher = entries(T, V, 3, g, none=0.0)
    index[bad, 1] = V if wrong == "V" else abs(wrong) + 10 ** 12  # below 0 would be no entry
    loss, lse, picked, dX, dW = distill_step(X, W, index, teacher, dloss)
    assert bool(torch.isnan(loss[bad])) and bool(torch.isnan(dX[bad]).all()) and bool(torch.isnan(dW).all())
    assert bool(torch.isfinite(loss[others]).all()) and bool(torch.isfinite(dX[others]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", PATHS)
def test_entries_named_twice_without_mass_and_strided(T, V, H, dtype):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 9)
    index, teacher = entries(T, V, 9, g)
    index[:, 3] = index[:, 1]
    index[:, 4] = index[:, 1]
    index[:, 5] = target
    teacher[:, 6] = -float("inf")
    teacher[:, 5] = torch.where(index[:, 5] >= 0, teacher[:, 5].clamp(min=-3), teacher[:, 5])
    run_distill(X, W, index[:, :7], teacher[:, :7], dloss, 0.9, 1.1, dtype)


@pytest.mark.parametrize("T,V,H", PATHS)
def test_fp32_powers_of_two_cancel(T, V, H):
    X, W, target, dloss, _ = inputs(T, V, H, "f32", 10)
    one = step(X, W, target, dloss)
    two = step(X * 2.0 ** 60, W * 2.0 ** -60, target, dloss)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert torch.equal(one[2], two[2] * 2.0 ** 60) and torch.equal(one[3], two[3] * 2.0 ** -60)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", PATHS)
def test_large_logits(T, V, H, dtype):
    # logits of some thousands: nothing overflows, the softmax is all but one-hot
    X, W, target, dloss, _ = inputs(T, V, H, dtype, 11)
    run_ce(X, W, target, dloss, 1000.0, dtype)
    run_ce(X, W, target, dloss, -1000.0, dtype)


@pytest.mark.parametrize("T,V,H", PATHS)
def test_fp32_wide_range(T, V, H):
    # rows of X and W from 1e-6 to 1e3 of each other, and values of 1e-12 among those of 1
    X, W, target, dloss, g = inputs(T, V, H, "f32", 12)
    X = X * torch.exp(torch.rand(T, 1, generator=g, device="cuda") * 8 - 6)
    X = torch.where(torch.rand(T, H, generator=g, device="cuda") < 0.2, X * 1e-12, X)
    W = W * torch.exp(torch.rand(V, 1, generator=g, device="cuda") * 8 - 7)
    run_ce(X, W, target, dloss * torch.exp(torch.rand(T, generator=g, device="cuda") * 12 - 10), 1.0, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", PATHS)
def test_streams_and_repeats_give_the_same_bits(T, V, H, dtype):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 13)
    index, teacher = entries(T, V, 6, g)
    one, two = step(X, W, target, dloss), distill_step(X, W, index, teacher, dloss)
    for _ in range(3):
        assert same(one, step(X, W, target, dloss)) and same(two, distill_step(X, W, index, teacher, dloss))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(X, W, target, dloss, stream=side), distill_step(X, W, index, teacher, dloss, stream=side)
    handle = step(X, W, target, dloss, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        inside = step(X, W, target, dloss)
    torch.cuda.current_stream().wait_stream(side)
    assert same(one, got[0]) and same(two, got[1]) and same(one, handle) and same(one, inside)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", PATHS)
def test_graph_replays(T, V, H, dtype):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 14)
    index, teacher = entries(T, V, 6, g)
    X = X.contiguous()

    def run():
        return step(X, W, target, dloss) + distill_step(X, W, index, teacher, dloss)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        run()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    base = X.clone()
    for i in range(4):
        X.copy_(base * (1 + 0.25 * i))
        target.copy_(target.roll(1))
        if i == 2:
            target[: T // 2 + 1] = -100
        eager = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(eager, captured), i


@pytest.mark.parametrize("dtype,T,V,H", [("bf16", 8192, 60001, 64), ("f32", 4100, 61000, 40)])
def test_several_pieces_of_the_vocabulary(dtype, T, V, H):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 15)
    target[torch.rand(T, generator=g, device="cuda") < 0.3] = -100
    run_ce(X, W, target, dloss, 1.0, dtype)
    index, teacher = entries(T, V, 3, g)
    run_distill(X, W, index, teacher, dloss, 0.5, 0.8, dtype)


# few whole large tiles, and enough vocabulary for middle ones in dX: in one piece, and in two
@pytest.mark.parametrize("dtype,T,V,H", [("bf16", 300, 20000, 1000), ("f32", 300, 20000, 1000),
                                         ("bf16", 1100, 300001, 100), ("f32", 1100, 150001, 100)])
def test_dx_in_middle_tiles(dtype, T, V, H):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 21)
    target[torch.rand(T, generator=g, device="cuda") < 0.3] = -100
    run_ce(X, W, target, dloss, 1.0, dtype)


# rows that end inside a slab: NaN stand behind them in the padding, and behind the last row's end
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("T,V,H", [(70, 144000, 8), (300, 70001, 72), (700, 13000, 1000), (1100, 140000, 136),
                                   (300, 2000, 72)])
def test_rows_that_end_inside_a_slab(T, V, H, pad):
    X, W, target, dloss, g = inputs(T, V, H, "bf16", 22, pad)
    memory = torch.full((V * W.stride(0) + 4096,), float("nan"), device="cuda", dtype=W.dtype)
    W = memory[:V * W.stride(0)].view(V, W.stride(0))[:, :H].copy_(W)
    target[torch.rand(T, generator=g, device="cuda") < 0.3] = -100
    run_ce(X, W, target, dloss, 1.0, "bf16")
    index, teacher = entries(T, V, 3, g)
    run_distill(X, W, index, teacher, dloss, 0.5, 0.8, "bf16")


# few tokens against 32 and against 64 vocabulary rows a workgroup, on both sides of the change
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", [(40, 8192, 130), (40, 8193, 130), (61, 12287, 77), (64, 12288, 512), (33, 20001, 64)])
def test_few_tokens_and_many_rows(T, V, H, dtype):
    X, W, target, dloss, g = inputs(T, V, H, dtype, 23, 3)
    target[torch.rand(T, generator=g, device="cuda") < 0.3] = -100
    run_ce(X, W, target, dloss, 1.0, dtype)
    index, teacher = entries(T, V, 5, g)
    run_distill(X, W, index, teacher, dloss, 0.5, 0.8, dtype)


# entries taken four to a wave, and added up over more lanes than a wave has
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H,K", [(60, 3000, 100, 701), (700, 2000, 77, 50), (2, 40, 33, 200)])
def test_many_entries(T, V, H, K, dtype):
    X, W, _, dloss, g = inputs(T, V, H, dtype, 24, 3)
    index, teacher = entries(T, V, K, g)
    index[1::7] = -1
    run_distill(X, W, index, teacher, dloss, 0.5, 0.8, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [7, 100])
def test_offsets_past_32_bits(dtype, T):
    V, H, ld = 70001, 64, 40000 if dtype == "bf16" else 20000
    X, W, target, dloss, _ = inputs(T, V, H, dtype, 16)
    wide = torch.empty(V, ld, device="cuda", dtype=DT[dtype])
    assert wide.numel() * wide.element_size() > 2 ** 32
    wide[:, :H] = W
    run_ce(X, wide[:, :H], target, dloss, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [20, 200])
def test_one_gradient_alone(dtype, T):
    X, W, target, dloss, g = inputs(T, 3000, 100, dtype, 17)
    loss, lse, dX, dW = step(X, W, target, dloss)
    a, none = sg.vocab_ce_grad(X, W, target, lse, dloss, want_dw=False)
    assert none is None and torch.equal(a, dX)
    none, b = sg.vocab_ce_grad(X, W, target, lse, dloss, want_dx=False)
    assert none is None and torch.equal(b, dW)
    with pytest.raises(ValueError):
        sg.vocab_ce_grad(X, W, target, lse, dloss, want_dx=False, want_dw=False)


@pytest.mark.parametrize("T", [20, 200])
def test_autograd_and_differences(T):
    """Against the formula (check) the other tests look; here against differences of the operators' own
    losses: L is smooth with third derivatives along a unit direction below 1, so a central difference
    with step h is off by h^2 + 2 * 1e-6 * L / h, L <= 20 its size: with h = 2^-5 below 4e-3 of the
    direction's norm sums here (directions are scaled to |d| = 1, gradients are of order 0.1 and more)."""
    X, W, target, _, g = inputs(T, 500, 60, "f32", 18)
    index, teacher = entries(T, 500, 5, g)
    weight = torch.rand(T, generator=g, device="cuda") / T

    def total(x, w):
        return ((sg.vocab_cross_entropy(x, w, target, 0.8) + sg.vocab_distillation(x, w, index, teacher, 0.7, 0.9))
                .double() * weight).sum()

    X, W = X.clone().requires_grad_(), W.clone().requires_grad_()
    total(X, W).backward()
    for t in (X, W):
        # along the gradient itself, where the derivative is largest: its norm
        d = t.grad / t.grad.norm()
        h = 2.0 ** -5
        with torch.no_grad():
            plus = total(*[(x + h * d) if x is t else x for x in (X, W)])
            minus = total(*[(x - h * d) if x is t else x for x in (X, W)])
        assert abs(float(plus - minus) / (2 * h) - float(t.grad.norm())) < 4e-3
    frozen = W.detach()
    x = X.detach().clone().requires_grad_()
    total(x, frozen).backward()
    assert torch.equal(x.grad, X.grad)


def test_refusals():
    X, W, target, dloss, g = inputs(8, 100, 32, "f32", 19)
    index, teacher = entries(8, 100, 3, g)
    loss, lse = sg.vocab_ce(X, W, target)
    bad = [
        (TypeError, lambda: sg.vocab_ce(X.half(), W, target)),
        (TypeError, lambda: sg.vocab_ce(X, W.bfloat16(), target)),
        (TypeError, lambda: sg.vocab_ce(X[0], W, target)),
        (TypeError, lambda: sg.vocab_ce(X, W, target.int())),
        (ValueError, lambda: sg.vocab_ce(X, W[:, :16], target)),
        (ValueError, lambda: sg.vocab_ce(X, W[:0], target)),
        (ValueError, lambda: sg.vocab_ce(X, W, target[:4])),
        (ValueError, lambda: sg.vocab_ce(X.t().contiguous().t(), W, target)),
        (ValueError, lambda: sg.vocab_ce(X[:1].expand(8, 32), W, target)),
        (ValueError, lambda: sg.vocab_ce(X.cpu(), W, target)),
        (ValueError, lambda: sg.vocab_ce(X, W, target.cpu())),
        (ValueError, lambda: sg.vocab_ce(X, W, target.repeat(2)[::2])),
        (ValueError, lambda: sg.vocab_ce_grad(X, W, target, lse[:3], dloss)),
        (TypeError, lambda: sg.vocab_ce_grad(X, W, target, lse, dloss.double())),
        (ValueError, lambda: sg.vocab_distill(X, W, index, teacher[:, :2])),
        (ValueError, lambda: sg.vocab_distill(X, W, index[:4], teacher[:4])),
        (ValueError, lambda: sg.vocab_distill(X, W, index[:, :0], teacher[:, :0])),
        (TypeError, lambda: sg.vocab_distill(X, W, index, teacher.double())),
        (ValueError, lambda: sg.vocab_distill_grad(X, W, index, teacher, lse, teacher[:, :2], dloss)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(str(i))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_example_learns(dtype):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "vocab_head.py")
    spec = importlib.util.spec_from_file_location("vocab_head_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=20, dtype=dtype, tokens=200, vocab=1000, hidden=128, say=lambda _: None)
    assert all(x == x for x in losses) and losses[-1] < 0.8 * losses[0]
