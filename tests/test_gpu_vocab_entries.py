"""GPU checks of distillation from teachers of many entries.  Bounds: vocab_checks.py."""
import pytest
import torch

import fp32_gemm_05_amd as sg
import vocab_checks as vc

pytestmark = pytest.mark.gpu


def problem(T, V, H, K, seed, rows=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda") * (1.5 / H ** 0.5)
    index = torch.randint(0, rows or V, (T, K), generator=g, device="cuda")
    index[torch.rand(T, K, generator=g, device="cuda") < 0.2] = -1
    teacher = torch.randn(T, K, generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    return X, W, index, teacher, dloss


def gradients(X, W, index, teacher, dloss):
    loss, lse, picked = sg.vocab_distill(X, W, index, teacher)
    dX, dW = sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss)
    return {"loss": loss, "lse": lse, "dX": dX, "dW": dW}


# either side of where entries are no longer compared each with each, and are no longer sorted in LDS; all
# rows named, or a few of them over and over
@pytest.mark.parametrize("T,V,H,K", [(3, 3000, 40, 192), (90, 3000, 40, 192), (3, 3000, 40, 193),
                                     (90, 3000, 40, 193), (70, 500, 33, 1500), (20, 9000, 40, 8192),
                                     (70, 9000, 40, 8193), (2, 30000, 24, 20011), (66, 2500, 24, 4100)])
@pytest.mark.parametrize("rows", [None, 2, 60])
def test_many_entries_of_a_token(T, V, H, K, rows):
    X, W, index, teacher, dloss = problem(T, V, H, K, K + T, rows)
    index[T // 2] = -1
    index[0] = 7
    got = gradients(X, W, index, teacher, dloss)
    keep = index >= 0
    counts = keep.any(1)
    q = torch.softmax(teacher.double().masked_fill(~keep, -float("inf")), 1)
    q = torch.where(counts[:, None], q, 0.0)
    r = vc.definition(X, W, 1.0, index, q, counts, dloss)
    vc.check_fp32_gradients(r, got)
    again = gradients(X, W, index, teacher, dloss)
    assert all(torch.equal(got[n], again[n]) for n in got)
    # an entry past the vocabulary is still its token's NaN
    index[1, K // 2] = V
    bad = gradients(X, W, index, teacher, dloss)
    others = torch.arange(T, device="cuda") != 1
    assert bool(torch.isnan(bad["dX"][1]).all()) and torch.equal(bad["dX"][others], got["dX"][others])


@pytest.mark.parametrize("T", [2, 80])
def test_time_grows_with_the_entries_not_their_square(T):
    def us(K):
        X, W, index, teacher, dloss = problem(T, 32768, 16, K, 3)
        loss, lse, picked = sg.vocab_distill(X, W, index, teacher)
        best = float("inf")
        for _ in range(5):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            sg.vocab_distill_grad(X, W, index, teacher, lse, picked, dloss)
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end))
        return best * 1000

    # 8 times the entries: 64 times the time if each is compared with each; sorting takes some 10 to 16
    small, large = us(2048), us(16384)
    print(f"T={T}: {small:.0f} us with 2048 entries, {large:.0f} us with 16384")
    assert large < 24 * small


@pytest.mark.parametrize("T", [5, 80])
@pytest.mark.parametrize("K", [300, 9000])
def test_graph_replays(T, K):
    X, W, index, teacher, dloss = problem(T, 2000, 40, K, T + K)

    def run():
        return gradients(X, W, index, teacher, dloss)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        run()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for i in range(4):
        index.copy_(index.roll(1, 0))
        index[i % T] = index[i % T].sort().values.flip(0)
        teacher.mul_(0.9)
        eager = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(eager[n], captured[n]) for n in eager), i
