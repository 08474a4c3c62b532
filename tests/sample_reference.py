"""Drawing tokens from rows of logits in 64 bits, row by row, and which tokens are right.  Runs on any device.

The kernels' exponentials exp(-x) are off by up to 2^-22 (their own last place and a product) + 2^-24 x (the rounding of
the logits' difference) of themselves, and their probabilities by half of 2^-40 of the largest one's.  The mean of x
weighted by exp(-x) is at most 1 + log(V) < 15, so a row's sums are off by less than 2^-20 + V 2^-41 of the whole.
Where a border (top_p's, min_p's, u's) lies nearer to a sum than `near` of the whole, either side of it is right:
`allowed` gives every token that is.
"""
import math

import torch


def value(setting, t):
    """A row's setting as the operator takes it, an fp32 value."""
    x = setting[t] if isinstance(setting, torch.Tensor) else torch.tensor(setting, dtype=torch.float32)
    return float(x)


def allowed(row, u, temperature, top_k, top_p, min_p):
    """The set of tokens that are right for a row of logits."""
    row = row.double().cpu()
    V = row.numel()
    u = float(u)
    top = float(row.max())
    if not math.isfinite(top) or bool(row.isnan().any()) or not 0 <= temperature < math.inf or any(
            math.isnan(x) for x in (u, top_p, min_p)):
        return {-1}
    if temperature == 0:
        return {int((row == top).nonzero()[0])}
    near = 2.0 ** -20 + V * 2.0 ** -41
    # -0 and 0 are equal; a stable sort keeps the lower index first
    order = torch.sort(-(row + 0.0), stable=True).indices
    p = ((row[order] - top) / temperature).exp()
    n = V if top_k <= 0 else min(V, top_k)
    n = min(n, int((row > -math.inf).sum()))
    p = p[:n]
    before = p.cumsum(0) - p
    total = float(p.sum())
    counts = {n}
    if top_p < 1:
        edge = top_p * total
        counts = {max(1, int((before < edge - near * total).sum())), max(1, int((before < edge + near * total).sum()))}
        counts = set(range(min(counts), max(counts) + 1)) if max(counts) - min(counts) < 50 else counts
    out = set()
    for c in counts:
        sizes = {c}
        if min_p > 0:
            # min_p goes by the logits: the border is exact but for the logarithm's own rounding
            sizes = {max(1, min(c, int((p >= min_p * (1 + s * 2.0 ** -45)).sum()))) for s in (-1, 1)}
        for size in sizes:
            chosen = order[:size].sort().values
            q = ((row[chosen] - top) / temperature).exp()
            sums = q.cumsum(0)
            whole = float(sums[-1])
            for shift in (-near, 0.0, near):
                at = int((sums <= (u + shift) * whole).sum())
                out.add(int(chosen[min(max(at, 0), size - 1)]))
    return out


def check(logits, u, token, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    assert token.dtype == torch.int64 and token.shape == u.shape
    rows, us, got = logits.float().cpu(), u.cpu(), token.tolist()
    settings = [s.cpu() if isinstance(s, torch.Tensor) else s for s in (temperature, top_k, top_p, min_p)]
    for t in range(rows.shape[0]):
        k = settings[1]
        k = int(k[t]) if isinstance(k, torch.Tensor) else k
        right = allowed(rows[t], us[t], value(settings[0], t), k, value(settings[2], t), value(settings[3], t))
        assert got[t] in right, (t, got[t], right)
