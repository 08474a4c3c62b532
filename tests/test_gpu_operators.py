"""GPU checks of the linear layer, the sampling and the gradient clipping as they are used: one after the other with
the vocabulary head, through autograd, on other streams, captured and replayed, at large offsets, with infinities."""
import math

import pytest
import torch

import fp32_gemm_05_amd as sg
import sample_reference
from linear_reference import ACTS, B, U, check_forward, check_gradients, slope, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def rand(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def model(g, T, H, F, V, dtype):
    return {"X": rand(g, T, H, dtype=dtype), "W1": rand(g, F, H, dtype=dtype, scale=H ** -0.5),
            "b1": rand(g, F, dtype=dtype, scale=0.2), "W2": rand(g, H, F, dtype=dtype, scale=F ** -0.5),
            "b2": rand(g, H, dtype=dtype, scale=0.2), "E": rand(g, V, H, dtype=dtype, scale=H ** -0.5)}


def loss_of(p, target, layer, head):
    h = layer(p["X"], p["W1"], p["b1"], None, "gelu")
    y = layer(h, p["W2"], p["b2"], p["X"], "none")
    return head(y, p["E"], target)


@pytest.mark.parametrize("T,H,F,V", [(40, 64, 200, 500), (300, 96, 260, 1000)])
def test_training_step(T, H, F, V):
    """Two layers on a residual stream, the vocabulary head, backward, clipping: against torch's own in 64 bits.

    fp32 throughout: each stage is off by some 10^-6 of its scale (its own tests bound it); chained through two layers and
    a softmax, gradients are held to 2^-14 of their tensor's norm."""
    g = gen(T)
    p = {k: v.requires_grad_() for k, v in model(g, T, H, F, V, F32).items()}
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::5] = -100
    loss = loss_of(p, target, sg.linear_layer, sg.vocab_cross_entropy)
    loss.sum().backward()

    def layer(x, w, b, r, act):
        y = x @ w.t() + b
        y = torch.nn.functional.gelu(y) if act == "gelu" else y
        return y if r is None else y + r

    def head(x, w, t):
        return torch.nn.functional.cross_entropy(x @ w.t(), t, ignore_index=-100, reduction="none")
    q = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    want = loss_of(q, target, layer, head)
    want.sum().backward()
    assert float((loss.double() - want).detach().abs().max()) < 2.0 ** -14
    grads = [v.grad for v in p.values()]
    for k in p:
        err = (p[k].grad.double() - q[k].grad).norm() / q[k].grad.norm()
        assert float(err) < 2.0 ** -14, (k, float(err))
    whole = math.sqrt(sum(float(v.grad.square().sum()) for v in q.values()))
    norm = sg.clip_grad_norm(grads, 0.5)
    assert abs(float(norm) / whole - 1) < 2.0 ** -14
    assert abs(float(sg.grad_norm(grads)) / 0.5 - 1) < 2.0 ** -14


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 50, 200])
def test_decoding_step(dtype, T):
    """Hidden states to logits in fp32, and tokens from them."""
    g = gen(T)
    p = model(g, T, 128, 300, 3000, dtype)
    y = sg.linear_act(sg.linear_act(p["X"], p["W1"], p["b1"], activation="silu"), p["W2"], p["b2"], p["X"])
    logits = sg.linear_act(y, p["E"], out_dtype=F32)
    assert logits.dtype == F32
    check_forward(y, p["E"], None, None, "none", logits)
    u = torch.rand(T, generator=g, device="cuda")
    s = dict(temperature=0.7, top_k=40, top_p=0.9, min_p=0.01)
    sample_reference.check(logits, u, sg.vocab_sample(logits, u, **s), **s)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", ACTS)
def test_autograd(dtype, name):
    g = gen(3)
    X, W, b, R = rand(g, 90, 40, dtype=dtype), rand(g, 70, 40, dtype=dtype, scale=0.2), rand(g, 70, dtype=dtype), rand(g, 90, 70, dtype=dtype)
    leaves = [t.requires_grad_() for t in (X, W, b, R)]
    dY = rand(g, 90, 70, dtype=dtype)
    Y = sg.linear_layer(*leaves, activation=name)
    dX, dW, db, dR = torch.autograd.grad(Y, leaves, dY)
    X, W, b, R = (t.detach() for t in leaves)
    check_forward(X, W, b, R, name, Y.detach())
    check_gradients(X, W, b, dY, name, dX, dW, db)
    assert torch.equal(dR, dY)
    # an upstream gradient without memory of its own, and one leaf alone
    Y = sg.linear_layer(X, leaves[1], None, None, name)
    one, = torch.autograd.grad(Y.sum(), [leaves[1]])
    check_gradients(X, W, None, torch.ones_like(dY), name, None, one,
                    (slope(X.double() @ W.double().t(), name)).sum(0).to(dtype))


@pytest.mark.parametrize("T", [8, 60, 200])
@pytest.mark.parametrize("name", ["none", "gelu", "gelu_tanh", "silu"])
def test_gradients_are_differences(T, name):
    """The directional derivative against central differences of the layer's own forward, in fp32.

    L(t) = sum dY * act((X + t V) W^T) along a direction V in X, W or the bias, d(t) = (L(t) - L(-t)) / 2t.  Its third
    derivative is at most A3 = sum |dY| 3 |z'|^3 + 6 |z'| |z''| + ..; with z'' = 0 along one operand that is
    sum |dY| 3 |z'|^3, as |act'''| < 3 for these; d is off by t^2 / 6 A3 and by the forward's errors, 2^-19 sum |dY| S
    at most, over t.  The gradient's own error is 2^-18 of the sum of its terms' magnitudes."""
    g = gen(T)
    N, H, t = 33, 47, 2.0 ** -6
    X, W, b, dY = rand(g, T, H), rand(g, N, H, scale=0.15), rand(g, N), rand(g, T, N)
    keep = name != "none"
    out = sg.linear_act(X, W, b, activation=name, keep=keep)
    grads = sg.linear_act_grad(X, W, dY, out[1] if keep else None, activation=name)
    for i, (operand, grad) in enumerate(zip((X, W, b), grads)):
        V = torch.randn(operand.shape, generator=g, device="cuda")

        def value(sign):
            moved = [X, W, b]
            moved[i] = operand + sign * t * V
            return float((sg.linear_act(*moved, activation=name).double() * dY.double()).sum())

        def along(X, W, V):
            return (V @ W.t() if i == 0 else X @ V.t() if i == 1 else V.expand(T, N)).double()
        dz = along(X, W, V)
        S = X.abs().double() @ W.abs().double().t() + b.abs().double() + t * dz.abs()
        a = dY.abs().double()
        tol = t * t / 6 * float((a * 3 * dz.abs() ** 3).sum()) + 2.0 ** -19 * float((a * S).sum()) / t
        tol += 2.0 ** -18 * float((a * 1.2 * along(X.abs(), W.abs(), V.abs())).sum())
        got = float((grad.double() * V.double()).sum())
        assert abs((value(1) - value(-1)) / (2 * t) - got) <= tol, (i, got, tol)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N,H", [(9, 130, 77), (100, 131, 1000), (300, 300, 90), (129, 520, 104)])
def test_infinities_and_nan_stay_in_their_rows(dtype, T, N, H):
    """At the ends of rows, where other elements stand in for what lies past them.  (Of up to 64 tokens a gradient, and
    of 17 to 64 an fp32 product, may make NaN of an infinity.)"""
    g = gen(7)
    X, W, dY = rand(g, T, H, dtype=dtype), rand(g, N, H, dtype=dtype), rand(g, T, N, dtype=dtype)
    clean = sg.linear_act(X, W, None)
    clean_dx, clean_dw, _ = sg.linear_act_grad(X, W, dY, want_dbias=False)

    def same(got, want, exactly=T > 64):
        """Infinities and NaN where 64 bits have them."""
        if exactly:
            assert bool((got.isnan() == want.isnan()).all()) and bool((got.isinf() == want.isinf()).all())
            assert bool((got.sign() == want.sign())[got.isinf()].all())
        else:
            assert bool((got.isfinite() == want.isfinite()).all())

    for value in (math.inf, -math.inf, math.nan):
        x = X.clone()
        x[T - 1, H - 1] = value
        y = sg.linear_act(x, W, None)
        same(y, x.double() @ W.double().t(), True)
        assert torch.equal(y[:-1], clean[:-1])
        dw = sg.linear_act_grad(x, W, dY, want_dx=False, want_dbias=False)[1]
        same(dw, dY.double().t() @ x.double())
        assert torch.equal(dw[:, :-1], clean_dw[:, :-1])
        w = W.clone()
        w[N - 1, H - 1] = value
        y = sg.linear_act(X, w, None)
        same(y, X.double() @ w.double().t(), True)
        assert torch.equal(y[:, :-1], clean[:, :-1])
        dx = sg.linear_act_grad(X, w, dY, want_dw=False, want_dbias=False)[0]
        same(dx, dY.double() @ w.double())
        assert torch.equal(dx[:, :-1], clean_dx[:, :-1])
        d = dY.clone()
        d[T - 1, N - 1] = value
        dx, dw, db = sg.linear_act_grad(X, W, d)
        same(dx, d.double() @ W.double())
        assert torch.equal(dx[:-1], clean_dx[:-1])
        same(dw, d.double().t() @ X.double())
        assert torch.equal(dw[:-1], clean_dw[:-1])
        same(db, d.double().sum(0))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N,H", [(40, 300, 70), (66, 9000, 3), (200, 1003, 257), (300, 64, 1024), (8191, 65, 33),
                                   (100, 20001, 63)])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_wanted_gradients_alone(dtype, T, N, H, name):
    """Each set of gradients has the bits that it has among all."""
    g = gen(T)
    X, W, dY = rand(g, T, H, dtype=dtype), rand(g, N, H, dtype=dtype, scale=H ** -0.5), rand(g, T, N, dtype=dtype)
    b = rand(g, N, dtype=dtype)
    Z = sg.linear_act(X, W, b, None, name, keep=True)[1]
    want = sg.linear_act_grad(X, W, dY, Z, name)
    check_gradients(X, W, b, dY, name, *want)
    for flags in range(1, 8):
        wanted = [bool(flags >> i & 1) for i in range(3)]
        got = sg.linear_act_grad(X, W, dY, Z, name, *wanted)
        for a, b, is_wanted in zip(got, want, wanted):
            assert a is None if not is_wanted else torch.equal(a, b), flags


def test_activations_far_out():
    """Slopes and values at the ends of the range: the limits, not NaN of an overflow on the way."""
    z = torch.tensor([-3e38, -1e20, -1e4, -60.0, -21.0, 0.0, 21.0, 60.0, 1e4, 1e20, 3e38, math.inf, math.nan], device="cuda")
    X, W = z[:, None].repeat(1, 1).contiguous(), torch.ones(1, 1, device="cuda")
    one = torch.ones_like(X)
    for T in (1, 10):  # few and many tokens
        x, d = X.repeat(T, 1), one.repeat(T, 1)
        for name in ("relu", "gelu", "gelu_tanh", "silu"):
            Y, Z = sg.linear_act(x, W, activation=name, keep=True)
            dX = sg.linear_act_grad(x, W, d, Z, activation=name)[0]
            n = len(z)
            if x.shape[0] > 64 or x.shape[0] <= 16:
                # small negative tails count as 0 here
                assert bool((Y[:n - 1, 0].nan_to_num(posinf=math.inf) >= -1e-6).all()) and bool(Y[n - 1].isnan())
                assert torch.equal(Y[6:n - 1, 0], z[6:n - 1]), name
                assert bool((dX[:4, 0].abs() < 1e-6).all()) and bool((dX[7:n - 2, 0] == 1).all()), (name, dX[:, 0])


def test_offsets_past_32_bits():
    g = gen(11)
    # results
    T, N, H = 66000, 33000, 8
    X, W, b = rand(g, T, H, dtype=BF16), rand(g, N, H, dtype=BF16), rand(g, N, dtype=BF16)
    Y = sg.linear_act(X, W, b, activation="relu")
    rows = torch.tensor([0, 1, 40000, T - 2, T - 1], device="cuda")
    check_forward(X[rows], W, b, None, "relu", Y[rows])
    dX, dW, db = sg.linear_act_grad(X, W, Y, Y, activation="relu")
    dz = torch.where(Y[rows] > 0, Y[rows], 0).double()
    within("dX", dX[rows], dz @ W.double(), 4 * B * (dz.abs() @ W.double().abs()))
    del Y, dX, dW
    # operands whose rows lie far apart
    wide = torch.empty(70, 1 << 24, device="cuda")
    x = wide[:, 5:45]
    x.copy_(rand(g, 70, 40))
    w = rand(g, 50, 40)
    check_forward(x, w, None, None, "none", sg.linear_act(x, w))
    check_gradients(x, w, None, rand(gen(1), 70, 50), "none", *sg.linear_act_grad(x, w, rand(gen(1), 70, 50)))
    del wide, x


def test_long_rows_of_logits():
    g = gen(12)
    T, V = 290, 1 << 23
    logits = torch.empty(T, V, device="cuda", dtype=BF16)
    logits.normal_(generator=g)
    u = torch.rand(T, generator=g, device="cuda")
    for s in (dict(), dict(top_p=0.3, temperature=0.6), dict(top_k=700)):
        token = sg.vocab_sample(logits, u, **s)
        assert bool(((token >= 0) & (token < V)).all())
        sample_reference.check(logits[-1:], u[-1:], token[-1:], **s)


def test_norm_of_a_long_tensor():
    n = (1 << 31) + 4099
    x = torch.full((n,), 0.5, device="cuda", dtype=BF16)
    x[-1] = 100.0
    want = math.sqrt(0.25 * (n - 1) + 1e4)
    assert abs(float(sg.grad_norm([x])) - want) <= 2 * U * want
    sg.clip_grad_norm([x], want / 4)
    assert float(x[-1]) == 25.0 and float(x[0]) == 0.125 and bool((x[:-1] == 0.125).all())


def operands():
    g = gen(5)
    p = model(g, 100, 64, 130, 900, F32)
    return {**p, "dY": rand(g, 100, 130), "logits": rand(g, 100, 900, scale=2), "u": torch.rand(100, generator=g, device="cuda"),
            "grads": [rand(g, 50, 33), rand(g, 7000, dtype=BF16), rand(g, 3)]}


def every_call(o):
    Y, Z = sg.linear_act(o["X"], o["W1"], o["b1"], activation="gelu", keep=True)
    dX, dW, db = sg.linear_act_grad(o["X"], o["W1"], o["dY"], Z, activation="gelu")
    few = sg.linear_act(o["X"][:5], o["W1"], o["b1"], activation="silu")
    fx, fw, fb = sg.linear_act_grad(o["X"][:5], o["W1"], o["dY"][:5])
    token = sg.vocab_sample(o["logits"], o["u"], temperature=0.8, top_k=30, top_p=0.9)
    other = sg.vocab_sample(o["logits"], o["u"], temperature=1.5, top_p=0.99, min_p=0.001)
    out = [torch.empty_like(t) for t in o["grads"]]
    norm = sg.clip_grad_norm(o["grads"], 0.7, out=out)
    return [Y, Z, dX, dW, db, few, fx, fw, fb, token, other, norm, sg.grad_norm(o["grads"])] + out


def fresh(o, seed):
    """New values in the same memory."""
    g = gen(seed)
    for k, t in o.items():
        for x in (t if isinstance(t, list) else [t]):
            x.copy_(torch.rand(x.shape, generator=g, device="cuda") if k == "u" else torch.randn(x.shape, generator=g, device="cuda"))


def test_graph_replays():
    o = operands()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        every_call(o)
    torch.cuda.current_stream().wait_stream(side)
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = every_call(o)
    with torch.cuda.graph(second, pool=graph.pool()):
        again = every_call(o)
    for seed in range(4):
        fresh(o, seed)
        graph.replay()
        first = [t.clone() for t in got]
        second.replay()
        torch.cuda.synchronize()
        want = every_call(o)
        for i, (a, b, c) in enumerate(zip(first, again, want)):
            assert torch.equal(a, c) and torch.equal(b, c), (seed, i)


@pytest.mark.parametrize("handle", [False, True])
def test_another_stream(handle):
    o = operands()
    want = every_call(o)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    s = stream.cuda_stream if handle else stream
    stream.wait_stream(torch.cuda.current_stream())
    Y, Z = sg.linear_act(o["X"], o["W1"], o["b1"], activation="gelu", keep=True, stream=s)
    dX, dW, db = sg.linear_act_grad(o["X"], o["W1"], o["dY"], Z, activation="gelu", stream=s)
    token = sg.vocab_sample(o["logits"], o["u"], temperature=0.8, top_k=30, top_p=0.9, stream=s)
    out = [torch.empty_like(t) for t in o["grads"]]
    norm = sg.clip_grad_norm(o["grads"], 0.7, out=out, stream=s)
    total = sg.grad_norm(o["grads"], stream=s)
    torch.cuda.current_stream().wait_stream(stream)
    for got, i in ((Y, 0), (Z, 1), (dX, 2), (dW, 3), (db, 4), (token, 9), (norm, 11), (total, 12)):
        assert torch.equal(got, want[i]), i
    for a, b in zip(out, want[13:]):
        assert torch.equal(a, b)


def test_captured_training_step():
    """Forward and backward through autograd in one graph, replayed with other values beside eager steps."""
    g = gen(1)
    p = model(g, 100, 64, 130, 50, F32)
    dY = rand(g, 100, 64)
    names = ["X", "W1", "b1", "W2", "b2"]

    def step():
        q = {k: p[k].detach().requires_grad_() for k in names}
        h = sg.linear_layer(q["X"], q["W1"], q["b1"], None, "silu")
        y = sg.linear_layer(h, q["W2"], q["b2"], q["X"], "none")
        return [y.detach(), *torch.autograd.grad(y, list(q.values()), dY)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        fresh({**{k: p[k] for k in names}, "dY": dY}, seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b), seed


def test_two_threads_at_once():
    """Calls of several host threads, each on a stream of its own."""
    import threading
    o = operands()
    want = every_call(o)
    torch.cuda.synchronize()
    results, errors = {}, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                results[i] = [every_call(o) for _ in range(3)]
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for calls in results.values():
        for got in calls:
            for a, b in zip(got, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N,H", [(1, 5, 3), (20, 70, 33), (60, 9, 500), (100, 131, 77), (300, 260, 264)])
def test_results_with_row_strides(dtype, T, N, H):
    """Results whose rows lie further apart than they are long, through the C entry points: what lies between the rows
    and behind the last one stays, and the rest is as without."""
    from fp32_gemm_05_amd import linear
    g = gen(T)
    X, W, dY = rand(g, T, H, dtype=dtype), rand(g, N, H, dtype=dtype, scale=H ** -0.5), rand(g, T, N, dtype=dtype)
    b, R = rand(g, N, dtype=dtype), rand(g, T, N, dtype=dtype)
    Y, Z = sg.linear_act(X, W, b, R, "gelu", keep=True)
    dX, dW, db = sg.linear_act_grad(X, W, dY, Z, "gelu")
    d, stream = int(dtype == BF16), torch.cuda.current_stream().cuda_stream

    def padded(rows, cols, pad):
        return torch.full((rows * (cols + pad) + 40,), 7.0, dtype=dtype, device="cuda")

    def unpadded(t, rows, cols, pad):
        whole = t[: rows * (cols + pad)].view(rows, cols + pad)
        assert bool((whole[:, cols:] == 7).all()) and bool((t[rows * (cols + pad):] == 7).all())
        return whole[:, :cols]
    y, z, x, w, s = padded(T, N, 3), padded(T, N, 8), padded(T, H, 1), padded(N, H, 5), padded(1, N, 0)
    work = [torch.empty(max(16, sg.linear_workspace(dtype, grad, T, N, H)), dtype=torch.uint8, device="cuda") for grad in (False, True)]
    linear._library.call("linear_act", d, d, T, N, H, X.data_ptr(), H, W.data_ptr(), H, b.data_ptr(), R.data_ptr(), N, 2,
                         y.data_ptr(), N + 3, z.data_ptr(), N + 8, work[0].data_ptr(), work[0].numel(), stream)
    assert torch.equal(unpadded(y, T, N, 3), Y) and torch.equal(unpadded(z, T, N, 8), Z)
    linear._library.call("linear_act_grad", d, T, N, H, X.data_ptr(), H, W.data_ptr(), H, dY.data_ptr(), N, z.data_ptr(),
                         N + 8, 2, x.data_ptr(), H + 1, w.data_ptr(), H + 5, s.data_ptr(), work[1].data_ptr(),
                         work[1].numel(), stream)
    assert torch.equal(unpadded(x, T, H, 1), dX) and torch.equal(unpadded(w, N, H, 5), dW)
    assert torch.equal(unpadded(s, 1, N, 0)[0], db)


def test_two_streams_at_once():
    o, streams = operands(), [torch.cuda.Stream() for _ in range(3)]
    want = every_call(o)
    torch.cuda.synchronize()
    results = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                results.append(every_call(o))
    torch.cuda.synchronize()
    for got in results:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
