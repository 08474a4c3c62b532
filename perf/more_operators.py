"""The operators around the vocabulary head as a user's program calls them, case by case, with their plain forms.

Three operators:

  linear   Y = act(X W^T + bias) + residual, and for training Z = X W^T + bias and the gradients
           dZ = dY * act'(Z), dX = dZ W, dW = dZ^T X, dbias = sum_t dZ[t];
  sample   one token per row of logits: z = logits / temperature, in the order of falling z (of equal
           ones the lower index first) the top_k first stay, of those each before which less than
           top_p of their mass lies, of those each of at least min_p times the first one's
           probability; the token is the first, by index, up to which more than u of the mass of what
           stays lies.  Temperature 0 takes the largest logit.  A row without a finite logit gives -1;
  clip     norm = sqrt(sum of squares over many tensors); every tensor times min(1, max_norm / (norm + 1e-6)).

`own` selects who computes: the plain form (elementary torch operations in 32 bits, in 64 where masses
are compared and where long sums are taken) or the framework's operators.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _linear(name, train, dtype, rows, out, hidden, act="none", bias=True, residual=False, wide=False, pad=0):
    c = {"op": "linear", "train": train, "dtype": dtype, "rows": rows, "out": out, "hidden": hidden, "act": act,
         "bias": bias, "residual": residual, "wide": wide, "pad": pad}
    return dict(c, name=name) if name else c


def _sample(name, dtype, rows, vocab, filters, per_row=False, spread=2.0, masked=0.0, pad=0):
    c = {"op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab, "filters": filters, "per_row": per_row,
         "spread": spread, "masked": masked, "pad": pad}
    return dict(c, name=name) if name else c


def _clip(name, clip, dtype, layers, hidden, vocab, max_norm=1.0, pad=0):
    c = {"op": "clip", "clip": clip, "dtype": dtype, "layers": layers, "hidden": hidden, "vocab": vocab,
         "max_norm": max_norm, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one generated token through a layer: the latency of a read of W
        _linear("linear 1 bf16", False, "bf16", 1, 4096, 1024, "silu"),
        # a few sequences' tokens in fp32, every size odd and the rows unaligned
        _linear("linear 37 f32 odd", False, "f32", 37, 5003, 777, "relu", residual=True, pad=3),
        # the logits of a batch of sequences, in fp32 for the sampling
        _linear("linear 64 bf16 logits", False, "bf16", 64, 32768, 1024, bias=False, wide=True),
        # an fp32 training step of ordinary size
        _linear("linear train 2048 f32", True, "f32", 2048, 4096, 1024, "gelu"),
        # a ragged training step, unaligned rows, on top of the residual stream
        _linear("linear train 777 bf16 odd", True, "bf16", 777, 5003, 1001, "silu", residual=True, pad=3),
        # the largest training step
        _linear("linear train 8192 bf16", True, "bf16", 8192, 8192, 4096, "gelu_tanh"),
        # one sequence's next token: latency
        _sample("sample 1 f32", "f32", 1, 32768, "top_k top_p"),
        # a batch being decoded, with each sequence's own settings
        _sample("sample 64 bf16 mixed", "bf16", 64, 131072, "mixed", per_row=True),
        # many sequences, flat distributions, odd rows, part of the vocabulary forbidden
        _sample("sample 1000 f32 odd", "f32", 1000, 50021, "top_p min_p", spread=2.5, masked=0.2, pad=3),
        # the norm of a small model's gradients, watched from step to step
        _clip("norm f32 small", False, "f32", 2, 256, 2000),
        # odd sizes, strided tensors, vectors in fp32 beside matrices in bf16
        _clip("clip mixed odd", True, "mixed", 6, 1001, 5003, pad=3),
        # a large model's gradients, some hundreds of tensors
        _clip("clip bf16 large", True, "bf16", 30, 1024, 65536),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    """Any operator, direction and type.  linear: 1 to 8192 rows, 64 to 8192 outputs, 64 to 4096 hidden, up to a
    fourth of the largest listed case's products in fp32; sample: 1 to 1024 rows of 500 to 131072 logits, up to
    1000 x 50021 in all, any filters; clip: 1 to 30 layers of 64 to 1500, up to the largest listed case's
    elements.  Half of the sizes are multiples of 64, the others as they fall, rows aligned and not."""
    even = rng.random() < 0.5
    pad = rng.choice((0, 0, 8, 3))

    def size(lo, hi):
        n = _log_uniform(rng, lo, hi)
        return max(64, n // 64 * 64) if even else n

    op = rng.choice(("linear", "linear", "sample", "clip"))
    while op == "linear":
        train = rng.random() < 0.5
        c = _linear(None, train, rng.choice(("f32", "bf16")), _log_uniform(rng, 1, 8192), size(64, 8192),
                    size(64, 4096), rng.choice(ACTIVATIONS), rng.random() < 0.7, rng.random() < 0.4, False, pad)
        c["wide"] = c["dtype"] == "bf16" and not train and rng.random() < 0.3
        most = 3 * 8192 * 8192 * 4096 // (4 if c["dtype"] == "f32" else 1)
        if c["rows"] * c["out"] * c["hidden"] * (3 if train else 1) <= most:
            return c
    while op == "sample":
        filters = rng.choice(("", "greedy", "top_k", "top_p", "min_p", "top_k top_p", "top_p min_p",
                              "top_k top_p min_p", "mixed"))
        c = _sample(None, rng.choice(("f32", "bf16")), _log_uniform(rng, 1, 1024), size(500, 131072), filters,
                    filters == "mixed" or rng.random() < 0.5, round(rng.uniform(0.5, 4.0), 2),
                    rng.choice((0.0, 0.0, round(rng.random() * 0.95, 2))), pad)
        if c["rows"] * c["vocab"] <= 1000 * 50021:
            return c
    while True:
        c = _clip(None, rng.random() < 0.7, rng.choice(("f32", "bf16", "mixed")), _log_uniform(rng, 1, 30),
                  size(64, 1500), size(500, 65536), rng.choice((0.5, 1.0, 1.0, 1e9)), pad)
        if sum(map(math.prod, _shapes(c))) <= sum(map(math.prod, _shapes(listed()[-1]))):
            return c


def _shapes(c):
    h = c["hidden"]
    layer = [(h, h)] * 4 + [(h,)] * 6 + [(4 * h, h), (4 * h,), (h, 4 * h), (h,)]
    return [(c["vocab"], h)] + layer * c["layers"] + [(h,)]


def _padded(x, pad):
    """x's rows `pad` elements further apart than they are long."""
    if not pad or x.dim() != 2:
        return x
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, device=x.device, dtype=x.dtype)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"linear": _prepare_linear, "sample": _prepare_sample, "clip": _prepare_clip}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_linear(c, g):
    """Normalised hidden states, weights that keep their scale, small biases; upstream gradients of a mean."""
    T, N, H = c["rows"], c["out"], c["hidden"]
    dtype = DTYPES[c["dtype"]]
    s = {"op": "linear", "act": c["act"], "train": c["train"],
         "X": _padded(_randn(g, T, H).to(dtype), c["pad"]),
         "W": _padded((_randn(g, N, H) / H ** 0.5).to(dtype), c["pad"]),
         "bias": (_randn(g, N) * 0.2).to(dtype) if c["bias"] else None,
         "out_dtype": torch.float32 if c["wide"] else dtype}
    s["residual"] = _padded(_randn(g, T, N).to(s["out_dtype"]), c["pad"]) if c["residual"] else None
    if c["train"]:
        s["dY"] = _padded((_randn(g, T, N) / T).to(dtype), c["pad"])
    return s


def _prepare_sample(c, g):
    """Logits of the given spread with some tokens that stand out, as a model's next tokens do; a part of the
    vocabulary forbidden for each row, for one row in fifty of many all of it."""
    T, V = c["rows"], c["vocab"]
    z = _randn(g, T, V) * c["spread"]
    lead = torch.randint(0, V, (T, 24), generator=g, device="cuda")
    rise = 4.0 + 8.0 * torch.rand(T, 24, generator=g, device="cuda")
    z.scatter_add_(1, lead, rise * torch.rand(T, 1, generator=g, device="cuda"))
    if c["masked"]:
        out = torch.rand(T, V, generator=g, device="cuda") < c["masked"]
        z.masked_fill_(out, -torch.inf)
        if T >= 50:
            z[torch.randperm(T, generator=g, device="cuda")[:T // 50]] = -torch.inf
    s = {"op": "sample", "logits": _padded(z.to(DTYPES[c["dtype"]]), c["pad"]),
         "u": torch.rand(T, generator=g, device="cuda"), "temperature": 0.8, "top_k": 0, "top_p": 1.0, "min_p": 0.0}
    f = c["filters"]
    if f == "greedy":
        s["temperature"] = 0.0
    if "top_k" in f:
        s["top_k"] = 50
    if "top_p" in f:
        s["top_p"] = 0.95
    if "min_p" in f:
        s["min_p"] = 0.02

    def pick(values, dtype=torch.float32):
        values = torch.tensor(values, device="cuda", dtype=dtype)
        return values[torch.randint(0, len(values), (T,), generator=g, device="cuda")]

    if f == "mixed":
        s.update(temperature=pick([0.0, 0.6, 0.8, 1.0, 1.3]), top_k=pick([0, 1, 20, 50, 1000, V], torch.int64),
                 top_p=pick([0.5, 0.9, 0.95, 0.99, 1.0]), min_p=pick([0.0, 0.0, 0.01, 0.1]))
    elif c["per_row"] and f != "greedy":
        s["temperature"] = pick([0.6, 0.8, 1.0, 1.3])
    return s


def _prepare_clip(c, g):
    """Gradients of tensors of a stack of layers, of scales as they come: some tensors a thousand times others."""
    grads = []
    for shape in _shapes(c):
        dtype = DTYPES["f32" if c["dtype"] == "f32" or (c["dtype"] == "mixed" and len(shape) == 1) else "bf16"]
        x = _randn(g, *shape)
        x *= 10 ** (-4.0 * torch.rand(1, generator=g, device="cuda"))
        grads.append(_padded(x.to(dtype), c["pad"]))
    s = {"op": "clip", "grads": grads, "max_norm": c["max_norm"], "align": 1 if c["pad"] % 8 else 64}
    if c["clip"]:
        # the gradients go on being added to, the optimizer takes the clipped ones, one flat buffer of each type
        s["flat"], s["clipped"] = _flat(grads, s["align"])
    return s


def _flat(tensors, align, dtype=None):
    """A buffer for each type among the tensors, and the places in it of tensors of their shapes."""
    at, sizes = [], {}
    for x in tensors:
        start = -(-sizes.get(x.dtype, 0) // align) * align
        at.append(start)
        sizes[x.dtype] = start + x.numel()
    flat = {t: torch.zeros(n, device="cuda", dtype=dtype or t) for t, n in sizes.items()}
    return list(flat.values()), [flat[x.dtype][a:a + x.numel()].view(x.shape) for x, a in zip(tensors, at)]


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def _plain_linear(s):
    dtype = s["X"].dtype
    x, w = s["X"].float(), s["W"].float()
    z = x @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"Y": y.to(s["out_dtype"])}
    if s["train"]:
        dz = s["dY"].float()
        if s["act"] != "none":
            dz = dz * _slope(z, s["act"])
        out["dX"], out["dW"] = (dz @ w).to(dtype), (dz.t() @ x).to(dtype)
        if s["bias"] is not None:
            out["dbias"] = dz.sum(0).to(dtype)
    return out


def _own_linear(s):
    import fp32_gemm_05_amd as sg
    keep = s["train"] and s["act"] != "none"
    y = sg.linear_act(s["X"], s["W"], s["bias"], s["residual"], activation=s["act"], out_dtype=s["out_dtype"],
                      keep=keep)
    y, z = y if keep else (y, None)
    out = {"Y": y}
    if s["train"]:
        out["dX"], out["dW"], dbias = sg.linear_act_grad(s["X"], s["W"], s["dY"], z, activation=s["act"],
                                                         want_dbias=s["bias"] is not None)
        if dbias is not None:
            out["dbias"] = dbias
    return out


def _column(value, rows, dtype=torch.float32):
    if not isinstance(value, torch.Tensor):
        value = torch.full((rows,), value, device="cuda", dtype=dtype)
    return value[:, None]


def _plain_sample(s):
    logits = s["logits"]
    T, V = logits.shape
    heat = _column(s["temperature"], T).double()
    z, order = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    greedy = heat == 0
    top = z[:, :1].double()
    mass = ((z.double() - top) / torch.where(greedy, 1.0, heat)).exp_()
    place = torch.arange(V, device="cuda")
    k = _column(s["top_k"], T, torch.int64)
    stays = place < torch.where(greedy, 1, torch.where(k <= 0, V, k))
    first = mass * stays
    before = first.cumsum(1) - first
    p = _column(s["top_p"], T).double()
    stays &= (before < p * first.sum(1, keepdim=True)) | (p >= 1)
    stays &= (mass >= _column(s["min_p"], T).double()) & (z > -torch.inf)
    kept = torch.zeros_like(mass).scatter_(1, order, mass * stays)
    total = kept.cumsum_(1)
    token = (total > s["u"][:, None].double() * total[:, -1:]).to(torch.uint8).argmax(1)
    return torch.where(torch.isfinite(top[:, 0]), token, -1)


def _own_sample(s):
    import fp32_gemm_05_amd as sg
    return sg.vocab_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                           min_p=s["min_p"])


def _plain_clip(s):
    total = torch.stack([x.float().square().sum(dtype=torch.float64) for x in s["grads"]]).sum()
    norm = total.sqrt().float()
    if "clipped" not in s:
        return norm
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    for x, out in zip(s["grads"], s["clipped"]):
        out.copy_(x.float() * scale)
    return [norm] + s["flat"]


def _own_clip(s):
    import fp32_gemm_05_amd as sg
    if "clipped" not in s:
        return sg.grad_norm(s["grads"])
    return [sg.clip_grad_norm(s["grads"], s["max_norm"], out=s["clipped"])] + s["flat"]


def run(state):
    if state["op"] == "linear":
        return _own_linear(state) if own else _plain_linear(state)
    if state["op"] == "sample":
        return _own_sample(state) if own else _plain_sample(state)
    return _own_clip(state) if own else _plain_clip(state)


def work(case):
    c = case
    if c["op"] == "linear":
        # in training X, W, dY and the residual read, Y, dX, dW and dbias written, once each
        T, N, H = c["rows"], c["out"], c["hidden"]
        size = 4 if c["dtype"] == "f32" else 2
        wide = 4 if c["wide"] else size
        moved = size * (T * H + N * H + N * c["bias"]) + wide * T * N * (1 + c["residual"])
        if c["train"]:
            moved += size * (T * N + T * H + N * H + N * c["bias"])
        return {"bytes": moved, "flops": 2 * T * N * H * (3 if c["train"] else 1)}
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * (4 if c["dtype"] == "f32" else 2) + 12),
                "flops": 4 * c["rows"] * c["vocab"]}
    moved = flops = 0
    for shape in _shapes(c):
        n = math.prod(shape)
        size = 4 if c["dtype"] == "f32" or (c["dtype"] == "mixed" and len(shape) == 1) else 2
        moved += n * size * (2 if c["clip"] else 1)
        flops += n * (3 if c["clip"] else 2)
    return {"bytes": moved + 4, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "sample": _exact_sample, "clip": _exact_clip}[case["op"]](s)


def _exact_linear(s):
    """torch's own layers in 64 bits, and their derivatives by torch."""
    train = s["train"]
    x, w = (s[n].double().requires_grad_(train) for n in ("X", "W"))
    b = None if s["bias"] is None else s["bias"].double().requires_grad_(train)
    f = torch.nn.functional
    act = {"none": lambda t: t, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh"),
           "silu": f.silu}[s["act"]]
    y = act(f.linear(x, w, b))
    if s["residual"] is not None:
        y = y + s["residual"].double()
    out = {"Y": y.detach()}
    if train:
        leaves = [x, w] if b is None else [x, w, b]
        out.update(zip(("dX", "dW", "dbias"), torch.autograd.grad(y, leaves, s["dY"].double())))
    return out


def _exact_sample(s):
    """Row by row: torch's softmax in 64 bits over what each filter has left, then the sum up to u."""
    logits = s["logits"]
    T, V = logits.shape

    def per_row(value):
        if isinstance(value, int):
            return [value] * T
        # settings are fp32 values, as the operator takes them
        return (value if isinstance(value, torch.Tensor) else torch.full((T,), value)).tolist()

    heat, k, p, least = (per_row(s[n]) for n in ("temperature", "top_k", "top_p", "min_p"))
    u = s["u"].double()
    tokens = []
    for t in range(T):
        row = logits[t].double()
        if not bool(torch.isfinite(row.max())):
            tokens.append(torch.tensor(-1, device="cuda"))
            continue
        if heat[t] == 0:
            tokens.append((row == row.max()).nonzero()[0, 0])
            continue
        value, index = torch.sort(row / heat[t], descending=True, stable=True)
        n = V if k[t] <= 0 else min(V, k[t])
        prob = torch.softmax(value[:n], 0)
        if p[t] < 1:
            n = max(1, int((prob.cumsum(0) - prob < p[t]).sum()))
        if least[t] > 0:
            n = max(1, min(n, int((prob >= least[t] * prob[0]).sum())))
        chosen = index[:n].sort().values
        prob = torch.softmax(row[chosen] / heat[t], 0)
        at = int((prob.cumsum(0) <= u[t] * prob.sum()).sum())
        tokens.append(chosen[min(at, n - 1)])
    return torch.stack(tokens)


def _exact_clip(s):
    each = [torch.linalg.vector_norm(x.double()) for x in s["grads"]]
    norm = torch.linalg.vector_norm(torch.stack(each))
    if "clipped" not in s:
        return norm
    scale = torch.minimum(torch.ones_like(norm), s["max_norm"] / (norm + 1e-6))
    flat, places = _flat(s["grads"], s["align"], torch.float64)
    for x, out in zip(s["grads"], places):
        torch.mul(x.double(), scale, out=out)
    return [norm] + flat
