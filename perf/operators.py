"""The vocabulary-head operators as a user's program calls them, case by case, with their plain forms.

Two operators over the logits z[t, v] = alpha * sum_h X[t, h] * W[v, h] of T tokens and a V-row
vocabulary matrix, neither of which keeps the T x V logits:

  cross entropy   loss[t] = lse[t] - z[t, target[t]], lse[t] = log(sum_v exp(z[t, v]));
  distillation    loss[t] = sum_k q[t, k] * (log(q[t, k]) - (z[t, index[t, k]] - lse[t])), with q the
                  softmax of the teacher's logits over the K entries that it gives for token t.

"score" cases run the forward pass; "train" cases the forward pass and the gradients of
sum_t dloss[t] * loss[t] with respect to X and W.  A token that carries the ignored target, or for
which the teacher gives no entry, has loss 0, lse 0 and gradient 0.

`own` selects who computes: the plain form (elementary torch operations in 32 bits) or the
framework's operators.
"""
import torch

own = False

IGNORED = -100
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(name, op, train, dtype, tokens, vocab, hidden, entries=0, ignored=0.0, pad=0):
    c = {"op": op, "train": train, "dtype": dtype, "tokens": tokens, "vocab": vocab, "hidden": hidden,
         "entries": entries, "ignored": ignored, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one generated token scored against the vocabulary: the latency of a read of W
        _case("ce score 1 bf16", "ce", False, "bf16", 1, 32768, 1024),
        # a short answer's log-probabilities in fp32, every size odd and the rows unaligned
        _case("ce score 61 f32 odd", "ce", False, "f32", 61, 50021, 777, pad=3),
        # perplexity of a batch of text
        _case("ce score 4096 bf16", "ce", False, "bf16", 4096, 32768, 4096),
        # the smallest training step: one short sequence, a small vocabulary
        _case("ce train 64 bf16", "ce", True, "bf16", 64, 8192, 512),
        # ragged fp32 step (characters or a small word list)
        _case("ce train 777 f32 ragged", "ce", True, "f32", 777, 5003, 1001),
        # an fp32 step of ordinary size
        _case("ce train 2048 f32", "ce", True, "f32", 2048, 32768, 2048),
        # fine-tuning on answers: the prompts' 60 % of the tokens do not count
        _case("ce train 8192 bf16 masked", "ce", True, "bf16", 8192, 32768, 2048, ignored=0.6),
        # the largest: a large vocabulary and hidden size
        _case("ce train 4096 bf16 large", "ce", True, "bf16", 4096, 131072, 4096),
        # a few tokens compared with a teacher during decoding
        _case("distill score 16 bf16", "distill", False, "bf16", 16, 65536, 2048, entries=16),
        # an fp32 student's step
        _case("distill train 1024 f32", "distill", True, "f32", 1024, 32768, 1024, entries=32),
        # odd sizes, unaligned rows, a quarter of the tokens without a teacher
        _case("distill train 1001 bf16 odd", "distill", True, "bf16", 1001, 50021, 1000, entries=20,
              ignored=0.25, pad=3),
        # a bf16 student's step of ordinary size
        _case("distill train 4096 bf16", "distill", True, "bf16", 4096, 65536, 4096, entries=64),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def _cost(c):
    return c["tokens"] * c["vocab"] * c["hidden"] * (3 if c["train"] else 1)


def draw(rng):
    """Any operator, direction and type; tokens 1 to 8192, vocabulary 500 to 131072, hidden 64 to 4096
    (half of the sizes multiples of 64, the others as they fall), up to 90 % ignored tokens, aligned and
    unaligned rows; never more work or more logits than the largest listed case."""
    most = 3 * 4096 * 131072 * 4096
    while True:
        tokens = _log_uniform(rng, 1, 8192)
        vocab = _log_uniform(rng, 500, 131072)
        hidden = _log_uniform(rng, 64, 4096)
        if rng.random() < 0.5:
            vocab, hidden = max(512, vocab // 64 * 64), hidden // 64 * 64
        op = rng.choice(("ce", "distill"))
        c = _case(None, op, rng.random() < 0.6, rng.choice(("f32", "bf16")), tokens, vocab, hidden,
                  entries=_log_uniform(rng, 1, 128) if op == "distill" else 0,
                  ignored=rng.choice((0.0, 0.0, round(rng.random() * 0.9, 2))), pad=rng.choice((0, 0, 8, 3)))
        if _cost(c) <= most and tokens * vocab <= 4096 * 131072:
            # in fp32 the plain form's own time bounds what a case may cost
            if c["dtype"] == "bf16" or _cost(c) <= most // 8:
                return c


def _counted(c):
    return c["tokens"] - int(c["tokens"] * c["ignored"])


def prepare(case, seed):
    """Hidden states of unit scale that lean towards their target's row of W (a trained model's target
    logits stand out), a W that gives logits of spread 1.5, and the upstream gradient of a weighted mean."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, V, H, pad = case["tokens"], case["vocab"], case["hidden"], case["pad"]
    dtype = DTYPES[case["dtype"]]

    def rows(x):
        if not pad:
            return x.to(dtype)
        wide = torch.zeros(x.shape[0], H + pad, device="cuda", dtype=dtype)
        wide[:, :H] = x
        return wide[:, :H]

    w = torch.randn(V, H, generator=g, device="cuda")
    w *= 1.5 / H ** 0.5
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda")
    lean = torch.rand(T, 1, generator=g, device="cuda") * 6
    x += lean * w[target] / 1.5
    n = _counted(case)
    out = torch.randperm(T, generator=g, device="cuda")[n:]
    state = {"X": rows(x), "W": rows(w)}
    dloss = (0.5 + torch.rand(T, generator=g, device="cuda")) / max(1, n)
    if case["train"]:
        state["dloss"] = dloss
    if case["op"] == "ce":
        target[out] = IGNORED
        state["target"] = target
        state["alpha"] = 1.0
        return state
    K = min(case["entries"], V)
    # distinct entries: the target, then steps through the vocabulary that never come round to it
    steps = torch.randint(1, max(2, V // K), (T, K), generator=g, device="cuda")
    steps[:, 0] = 0
    index = (target[:, None] + torch.cumsum(steps, 1)) % V
    teacher = torch.randn(T, K, generator=g, device="cuda") * 0.5 - 0.1 * torch.arange(K, device="cuda")
    teacher[:, 0] += 2.0
    given = torch.randint(1, K + 1, (T, 1), generator=g, device="cuda")
    given[out] = 0
    index[torch.arange(K, device="cuda") >= given] = -1
    state["index"], state["teacher"] = index, teacher
    state["alpha"] = 0.5  # temperature 2 on both sides
    return state


def _logits(s):
    x, w = s["X"].float(), s["W"].float()
    z = (x @ w.t()).mul_(s["alpha"])
    top = z.max(1, keepdim=True).values
    total = (z - top).exp_().sum(1, keepdim=True)
    return x, w, z, top + total.log()


def _gradients(s, x, w, d):
    dtype = s["X"].dtype
    return (d @ w).to(dtype), (d.t() @ x).to(dtype)


def _plain_ce(s):
    x, w, z, lse = _logits(s)
    counts = s["target"] != IGNORED
    at = torch.where(counts, s["target"], 0)[:, None]
    loss = torch.where(counts, (lse - z.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": torch.where(counts, lse[:, 0], 0.0)}
    if "dloss" in s:
        scale = torch.where(counts, s["dloss"] * s["alpha"], 0.0)[:, None]
        d = z.sub_(lse).exp_()
        d.scatter_add_(1, at, torch.full_like(lse, -1.0))
        out["dX"], out["dW"] = _gradients(s, x, w, d.mul_(scale))
    return out


def _plain_distill(s):
    x, w, z, lse = _logits(s)
    given = s["index"] >= 0
    counts = given.any(1)
    at = torch.where(given, s["index"], 0)
    t = torch.where(given, s["teacher"] * s["alpha"], -torch.inf)
    top = torch.where(counts, t.max(1).values, 0.0)[:, None]
    mass = torch.where(given, (t - top).exp(), 0.0)
    total = torch.where(counts[:, None], mass.sum(1, keepdim=True), 1.0)
    q = mass / total
    log_q = torch.where(given, t - top - total.log(), 0.0)
    loss = (q * torch.where(given, log_q - z.gather(1, at) + lse, 0.0)).sum(1)
    out = {"loss": loss, "lse": torch.where(counts, lse[:, 0], 0.0)}
    if "dloss" in s:
        scale = torch.where(counts, s["dloss"] * s["alpha"], 0.0)[:, None]
        d = z.sub_(lse).exp_()
        d.scatter_add_(1, at, -q)
        out["dX"], out["dW"] = _gradients(s, x, w, d.mul_(scale))
    return out


def _own_ce(s):
    import fp32_gemm_05_amd as sg
    loss, lse = sg.vocab_ce(s["X"], s["W"], s["target"], alpha=s["alpha"], ignore_index=IGNORED)
    out = {"loss": loss, "lse": lse}
    if "dloss" in s:
        out["dX"], out["dW"] = sg.vocab_ce_grad(s["X"], s["W"], s["target"], lse, s["dloss"], alpha=s["alpha"],
                                                ignore_index=IGNORED)
    return out


def _own_distill(s):
    import fp32_gemm_05_amd as sg
    loss, lse, picked = sg.vocab_distill(s["X"], s["W"], s["index"], s["teacher"], alpha=s["alpha"],
                                         teacher_alpha=s["alpha"])
    out = {"loss": loss, "lse": lse}
    if "dloss" in s:
        out["dX"], out["dW"] = sg.vocab_distill_grad(s["X"], s["W"], s["index"], s["teacher"], lse, picked,
                                                     s["dloss"], alpha=s["alpha"], teacher_alpha=s["alpha"])
    return out


def run(state):
    if "target" in state:
        return _own_ce(state) if own else _plain_ce(state)
    return _own_distill(state) if own else _plain_distill(state)


def work(case):
    """The products of the tokens that count with W (and, in training, the two products of their
    gradients), X and W read once, the outputs written once."""
    T, V, H, n = case["tokens"], case["vocab"], case["hidden"], _counted(case)
    size = 4 if case["dtype"] == "f32" else 2
    read = size * (n * H + V * H) + (8 * T if case["op"] == "ce" else 12 * T * case["entries"])
    wrote = 8 * T
    if case["train"]:
        read += 4 * T
        wrote += size * (T * H + V * H)
    return {"bytes": read + wrote, "flops": 2 * n * V * H * (3 if case["train"] else 1)}


def exact(case, seed):
    """The same by torch's own log-softmax and its derivative, in 64 bits, from the definition."""
    s = prepare(case, seed)
    train = "dloss" in s
    x = s["X"].double().requires_grad_(train)
    w = s["W"].double().requires_grad_(train)
    logits = torch.nn.functional.linear(x, w) * s["alpha"]
    logp = torch.log_softmax(logits, 1)
    if "target" in s:
        counts = s["target"] != IGNORED
        loss = torch.nn.functional.nll_loss(logp, s["target"], ignore_index=IGNORED, reduction="none")
    else:
        counts = s["index"][:, 0] >= 0
        keep = s["index"] >= 0
        scores = (s["teacher"].double() * s["alpha"]).masked_fill(~keep, -1e300)
        q = torch.softmax(scores, 1) * keep
        student = torch.gather(logp, 1, s["index"].clamp(min=0))
        loss = (torch.special.xlogy(q, q) - q * student).sum(1)
    lse = (logits.detach()[:, 0] - logp.detach()[:, 0]) * counts
    out = {"loss": loss.detach(), "lse": lse}
    if train:
        out["dX"], out["dW"] = torch.autograd.grad((loss * s["dloss"].double()).sum(), (x, w))
    return out
