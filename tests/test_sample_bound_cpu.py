"""CPU check of the sampling's stated precision: its exponential's fp32 arithmetic (weight_of in kernel_sample.hpp), step by
step in numpy, against 64 bits and the bound that sample.h states for it."""
import math
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
f32 = np.float32


def stated_bound():
    text = re.sub(r"\s*\n \*\s*", " ", open(os.path.join(ROOT, "include", "sample.h")).read())
    a, b = re.search(r"largest logit is off by up to 2\^-(\d+) \+ 2\^-(\d+) x of itself", text).groups()
    return 2.0 ** -int(a), 2.0 ** -int(b)


def weights(logit, top, temperature):
    exact = 1.4426950408889634 / float(temperature)
    c = f32(exact)
    if float(c) > exact:
        c = np.nextafter(c, f32(0))
    c_low = max(f32(exact - float(c)), c * f32(2.0 ** -40))
    d = logit - top
    # a fused multiply and add: the product of two fp32 numbers is exact in 64 bits
    e = (d.astype(np.float64) * float(c) + (d * c_low).astype(np.float64)).astype(f32)
    return np.exp2(e.astype(np.float64))


@pytest.mark.parametrize("temperature", [1.0, 0.7, 0.8, 1.3, 2.3, 0.05, 40.0])
@pytest.mark.parametrize("height", [0.0, 6.0, 1000.0])
def test_exponentials_within_the_stated_bound(temperature, height):
    """Distances up to 28, past which a token is not drawn.  The last place of the hardware's exponential, 2^-23, is left
    to the bound's constant: the emulated part has to stay within the rest."""
    rng = np.random.default_rng(int(height) + int(1000 * temperature))
    t = f32(temperature)
    n = 400000
    top = rng.normal(0, height + 1e-3, n).astype(f32)
    logit = np.minimum((top - rng.uniform(0, 28, n) * float(t)).astype(f32), top)
    x = (top.astype(np.float64) - logit.astype(np.float64)) / float(t)
    off = np.abs(weights(logit, top, t) * np.exp(x) - 1)
    constant, slope = stated_bound()
    over = off / (constant - 2.0 ** -23 + slope * x)
    assert over.max() <= 1, over.max()


def test_the_bound_is_the_sum_of_the_roundings():
    """The logits' difference and the exponent are rounded once each, by half a step, 2^-24 of x each; the exponential has its
    last place, 2^-23, and a product another half step."""
    constant, slope = stated_bound()
    assert slope == 2 * 2.0 ** -24 and constant >= 2.0 ** -23 + 2.0 ** -24
    # the weighted mean of x is at most 1 + log V: what a row's sums may be off by, for any V
    assert constant + slope * (1 + math.log(1 << 23)) < 2.0 ** -18
