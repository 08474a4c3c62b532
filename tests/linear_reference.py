"""The linear layer with an epilogue in 64 bits, and what its results may be off by.  Runs on any device.

Tolerances (derived, not tuned).  u = 2^-24 is half a step of fp32, b = 2^-8 the largest relative rounding of bf16.

Z is a sum of H products and a bias: |error| <= (H + 4) u S, S = sum |x w| + |bias| (three bf16 parts, of 17 to 64
fp32 tokens, hold a value to 2^-24 and leave out products below 2^-24 of the whole: 4 u S more).  An activation
passes an error on times its largest slope, 1.13, and adds its own: exponentials, reciprocals and the normal tail's
polynomial are off by up to 2^-20 relative, an exponent of -t^2 / 2 or -2 w by a few u of itself, which at the places
where it is large leaves a value that is small.  So |act error| <= 1.2 (H + 8) u S + 2^-19 |z| where z > -20, and the residual and Y's
rounding add u (fp32) or b (bf16) times the magnitudes.

dZ = dY act'(Z): with Z held in bf16 its slope is off by act'' b |z| at most, act'' <= 1.13, and 2^-19 for its own
arithmetic; dZ is rounded once in bf16 (b).  A gradient is a sum of n such terms: (n + 4) u A on top, A the sum of the
terms' magnitudes, and one rounding of the result (b).
"""
import math

import torch

U, B = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, 0.0, z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "none":
        return torch.ones_like(z)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = z.clamp(-40, 40)
    if name == "gelu_tanh":
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (c + 0.044715 * c ** 3))
        return s + s * (1 - s) * 2 * math.sqrt(2 / math.pi) * c * (1 + 3 * 0.044715 * c * c)
    s = torch.sigmoid(c)
    return s * (1 + c * (1 - s))


def forward(X, W, bias, residual, name):
    """Z, Y and the bounds of Z's and Y's errors before Y's own rounding."""
    x, w = X.double(), W.double()
    z, S = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, S = z + bias.double(), S + bias.double().abs()
    y = act(z, name)
    tz = (X.shape[1] + 8) * U * S
    ty = 1.2 * tz + 2.0 ** -19 * y.abs() + 2.0 ** -22 * (z.abs() if name not in ("none", "relu") else 0.0)
    if residual is not None:
        y = y + residual.double()
        ty = ty + U * y.abs()
    return z, y, tz, ty


def rounded(t, dtype):
    return B if dtype == torch.bfloat16 else U


def within(name, got, want, tol):
    """Every element within its tolerance; a NaN where there should be none fails."""
    bad = ~((got.double() - want).abs() <= tol + 1e-37)
    if bool(bad.any()):
        at = bad.nonzero()[:4].tolist()
        worst = ((got.double() - want).abs() / (tol + 1e-37)).nan_to_num(float("inf")).max()
        raise AssertionError((name, int(bad.sum()), at, float(worst)))


def check_forward(X, W, bias, residual, name, Y, Z=None):
    z, y, tz, ty = forward(X, W, bias, residual, name)
    within("Y", Y, y, ty + rounded(Y, Y.dtype) * (y.abs() + ty))
    if Z is not None:
        assert Z.dtype == X.dtype
        within("Z", Z, z, tz + rounded(Z, Z.dtype) * (z.abs() + tz))


def check_gradients(X, W, bias, dY, name, dX, dW, dbias):
    """Against the formula from the unrounded Z."""
    half = X.dtype == torch.bfloat16
    z, _, tz, _ = forward(X, W, bias, None, name)
    x, w, dy = X.double(), W.double(), dY.double()
    s = slope(z, name)
    dz = dy * s
    if name == "relu":
        # the slope jumps at 0: where Z's rounding may cross it, either side is right
        off = torch.where(z.abs() <= tz, dy.abs(), 0.0)
    elif name == "none":
        off = torch.zeros_like(dz)
    else:
        off = dy.abs() * (1.2 * (tz + (B * z.abs() if half else U * z.abs())) + 2.0 ** -19)
    own = B if half else U
    T, N = dy.shape
    within("dbias", dbias, dz.sum(0), off.sum(0) + (T + 4) * U * dz.abs().sum(0) + own * dz.abs().sum(0))
    each = off + own * (dz.abs() + off)  # of dZ as it enters the products
    for what, got, want, tol, A, n in (("dX", dX, dz @ w, each @ w.abs(), dz.abs() @ w.abs(), N),
                                       ("dW", dW, dz.t() @ x, each.t() @ x.abs(), dz.abs().t() @ x.abs(), T)):
        if got is not None:
            assert got.dtype == X.dtype
            within(what, got, want, tol + (n + 8) * U * A + own * (want.abs() + tol))
