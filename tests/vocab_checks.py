"""The vocabulary-head operators' definition in float64, the plain form in float32, and checks that see NaN and
lost digits.  Runs on any device.

Rows of results are compared in their 2-norm.  With u = 2^-24, H the hidden size and A the sum of a
result's terms in absolute value, E stands for the relative error that fp32 gives exp(z - lse):

  a logit is a sum of H products; each of its roundings is off by at most u times a partial sum, and
  partial sums of terms of either sign stay below |z| + 4 R, R the root of the sum of the squared terms.
  H such errors, each at most u (|z| + 4 R) and of either sign, add up to less than 4 sqrt(H) times that
  in all but one of 10^4 cases; lse, exp and the difference add a few u (|z| + |lse| + 2).
  E = 4 sqrt(H + 16) u (max |z| + |lse| + 4 R + 2).

A gradient's row is then off by at most (E + (4 sqrt(n) + 8) u) A in norm, n its number of terms, the 8 for
the operands' and D's own roundings (two fp16 planes are off by up to 2^-23 each), plus the planes' floor: D's entries are held
to 2^-40 of 1 (times |s|, s = alpha * dloss), W to 2^-40 of its largest value, s * X of dW to 2^-40 of its
largest; a rounding and its mirror in the other operand make that 2^-39.
"""
import torch

U = 2.0 ** -24


def definition(X, W, alpha, index, q, counts, dloss, dtype=torch.float64):
    """Loss, lse, D and the gradients in `dtype`, for targets given as entries with weights q (T x K), and what
    the bounds need."""
    x = torch.where(counts[:, None], X.to(dtype), 0.0)
    w = W.to(dtype)
    z = alpha * (x @ w.t())
    top = z.max(1, keepdim=True).values
    lse = (top + (z - top).exp().sum(1, keepdim=True).log())[:, 0]
    keep = index >= 0
    at = index.clamp(min=0)
    q = q.to(dtype)
    y = torch.zeros_like(z).scatter_add_(1, at, q * keep)
    loss = torch.where(keep & (q > 0), q * (q.clamp(min=1e-30).log() - z.gather(1, at) + lse[:, None]), 0.0).sum(1)
    s = torch.where(counts, alpha * dloss.to(dtype), 0.0)[:, None]
    p = (z - lse[:, None]).exp()
    d = s * (p - y)
    a = s.abs() * (p + y)
    r = abs(alpha) * (x.square() @ w.square().t()).max(1).values.sqrt()
    e = 4 * (X.shape[1] + 16) ** 0.5 * U * (z.abs().max(1).values + lse.abs() + 4 * r + 2)
    zero = torch.zeros((), dtype=dtype, device=X.device)
    sx = (s * x).abs()
    scale = r + z.abs().max(1).values + lse.abs() + 2
    return {"scale": scale, "SX": scale[:, None] * (a @ w.abs()), "SW": (a * scale[:, None]).t() @ x.abs(),
            "QX": (d.square() @ w.square()).sqrt(), "QW": (d.square().t() @ x.square()).sqrt(),
            "loss": torch.where(counts, loss, zero), "lse": torch.where(counts, lse, zero), "p": p, "d": d, "s": s,
            "E": e, "dX": d @ w, "dW": d.t() @ x, "AX": a @ w.abs(), "AW": a.t() @ x.abs(),
            # the part of dX's and dW's terms that a token's own E enters
            "EX": e[:, None] * (a @ w.abs()), "EW": (a * e[:, None]).t() @ x.abs(),
            "GX": 2.0 ** -39 * (s.abs() * w.abs().sum(0) + a.sum(1, keepdim=True) * w.abs().max()),
            "GW": 2.0 ** -39 * (sx.sum(0) + (p + y).sum(0)[:, None] * sx.max())}


def rows_within(name, got, want, bound):
    """Every row's error in norm within its bound; a NaN or an infinity fails."""
    err = (got.double() - want.double()).norm(dim=-1)
    bound = bound.double().norm(dim=-1)
    bad = ~(err <= bound + 1e-37)
    assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:4].flatten().tolist(),
                                 float((err / (bound + 1e-300)).nan_to_num(float("inf")).max()))


def check_fp32_gradients(r, got, tokens=slice(None), vocabulary=slice(None)):
    """dX and dW of an fp32 call, row by row, for the named rows."""
    n_x, n_w = r["p"].shape[1], r["p"].shape[0]
    for name, n, rows in (("dX", n_x, tokens), ("dW", n_w, vocabulary)):
        of = name[1]
        bound = r["E" + of] + (4 * n ** 0.5 + 8) * U * r["A" + of] + r["G" + of]
        rows_within(name, got[name][rows], r[name][rows], bound[rows])


def block_norms(x, rows=64):
    """The root mean square of blocks of `rows` values."""
    n = -(-x.shape[0] // rows)
    return torch.nn.functional.pad(x, (0, n * rows - x.shape[0])).view(n, rows).square().sum(1).sqrt()


def check_digits(r, plain, got, dtype, names=("loss", "lse", "dX", "dW")):
    """Errors as small as the arithmetic's own, so that a lost low part of an operand shows: twice the plain
    float32 form's (`plain`), and 16 u of the scale of what a value is computed from -- R, the largest logit and lse
    for the exponents, and that times a gradient's terms.  The planes' roundings make 1 u of R of a logit in
    the mean, those of exp, log and their arguments 3 u; a row of dW may hang on one logit, of which one in 10^6 is off by
    four times the mean.  (fp16 alone, without a low part, is off by 2000 u of R.)  In bf16, D and s X are
    rounded, each by at most b = 2^-8 and independently, so their n terms' errors add up like their squares
    (Q), and the result is rounded once: b (2 Q + |result|) more.  In norm by row; loss and lse by blocks of 64
    tokens."""
    b = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for name in names:
        err = got[name].double() - r[name].double()
        own = (plain[name].double() - r[name].double()).abs()
        if name in ("loss", "lse"):
            err, own, rest = (block_norms(v) for v in (err.abs(), own, 16 * U * r["scale"].double()))
        else:
            of = name[1]
            rest = 16 * U * r["S" + of] + b * (2 * r["Q" + of] + r[name].abs()) + r["G" + of]
            err, own, rest = (v.double().norm(dim=-1) for v in (err, own, rest))
        bad = ~(err <= 2 * own + rest + 1e-37)
        assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:4].flatten().tolist(),
                                     float((err / (2 * own + rest + 1e-300)).nan_to_num(float("inf")).max()))
