"""Linear layers whose results are known to the last bit.  Runs on any device.

X, W, dY, bias and residual hold whole numbers from -2 to 2, so every product and every sum of up to 2^20 of them, in any order
and cut anywhere, is a whole number that fp32 holds; parts of bf16 hold them too.  Each result is that number rounded
once to its type.  An activation's slope is made 0 or 1 exactly by the Z that is handed to the gradient: far out every one of
them is.  A row, a column or a partial sum that is lost, counted twice or rounded on the way shows.
"""
import torch

OFF, ON = -128.0, 32.0  # of Z: slopes 0 and 1 of every activation


def whole(g, *shape, dtype, device, pad=0):
    x = torch.randint(-2, 3, shape, generator=g, device=device).to(dtype)
    if not pad:
        return x
    wide = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=dtype, device=device)
    wide[:, :shape[1]] = x
    return wide[:, :shape[1]]


def inputs(T, N, H, dtype, device, pad=0, seed=0):
    g = torch.Generator(device=device).manual_seed(seed + 31 * T + N)
    p = {"X": whole(g, T, H, dtype=dtype, device=device, pad=pad), "W": whole(g, N, H, dtype=dtype, device=device, pad=pad),
         "bias": whole(g, N, dtype=dtype, device=device), "residual": whole(g, T, N, dtype=dtype, device=device, pad=pad),
         "dY": whole(g, T, N, dtype=dtype, device=device, pad=pad)}
    on = torch.rand(T, N, generator=g, device=device) < 0.7
    p["Z"] = torch.where(on, ON, OFF).to(dtype)
    return p


def forward(p, name, residual=True):
    """Y and Z, of "none" and "relu"."""
    z = p["X"].double() @ p["W"].double().t() + p["bias"].double()
    y = z.clamp(min=0) if name == "relu" else z
    return (y + p["residual"].double() if residual else y), z


def gradients(p, name):
    dz = p["dY"].double() * ((p["Z"] == ON).double() if name != "none" else 1.0)
    return dz @ p["W"].double(), dz.t() @ p["X"].double(), dz.sum(0)


def equal(got, want, what=""):
    """The bits of `want` rounded once."""
    assert got.shape == want.shape
    bad = got.double() != want.to(got.dtype).double()  # (whole numbers below 2^24: to fp32 exactly, so rounded once)
    bad |= got.isnan()
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist())
