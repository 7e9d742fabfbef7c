"""The normal tail's polynomial of the gated feed-forward kernels, evaluated in
fp32 on the CPU as the kernel does (Horner's rule with one rounding a step is at
least as exact as numpy's two), against erfc in fp64.

Bound: the fit's own error 6.2e-8 of q and |g| q, plus fp32's: P is about -1 to
-24, so its rounding errs by at most 2^-24 * 8 steps of |P| relative to 2^P,
whose product with q stays below 5e-8."""
import os
import re

import numpy as np
from scipy.special import erfc

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "diffusion_unet_attention_b200", "csrc",
                   "gated_ff.cuh")


def constants():
    text = open(SRC).read()
    c = [np.float32(re.search(rf"kTail{k} = ([-\d.e]+)f", text).group(1)) for k in range(8)]
    return c, np.float32(re.search(r"kTailBound = ([\d.]+)f", text).group(1))


def test_tail_and_gelu():
    c, bound = constants()
    g = np.concatenate([np.linspace(-12, 12, 400001), [0.0, -0.0, 1e-30, -1e-30, 5.6, -5.6, 100, -100]]).astype(np.float32)
    m = np.maximum(-np.abs(g), -bound)
    y = np.full_like(m, c[7])
    for k in range(6, -1, -1):
        y = (y * m + c[k]).astype(np.float32)
    q = np.exp2(y.astype(np.float64)).astype(np.float32)
    want = 0.5 * erfc(np.abs(g.astype(np.float64)) / np.sqrt(2))
    assert np.abs(q - want).max() <= 1.2e-7
    assert q[np.abs(g) >= bound].max() <= 2.0 ** -46      # gates past the clamp: the activation is g or 0
    gelu = np.maximum(g, 0).astype(np.float64) + m.astype(np.float64) * q
    exact = g.astype(np.float64) * 0.5 * erfc(-g.astype(np.float64) / np.sqrt(2))
    assert np.abs(gelu - exact).max() <= 1.2e-7


def test_constants_are_the_fits():
    import importlib.util
    spec = importlib.util.spec_from_file_location("gelu_tail_fit", os.path.join(os.path.dirname(SRC), "gelu_tail_fit.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    err, p = fit.fit()
    assert err <= 7e-8
    c, bound = constants()
    assert bound > fit.BOUND
    # another linear algebra library may level the errors a little differently:
    # the same polynomial to 1e-7 of q where it matters
    x = np.linspace(0, fit.BOUND, 2001)
    a, b = (np.polynomial.polynomial.polyval(-x, np.asarray(v, np.float64)) for v in (c, p))
    assert (np.abs(2 ** a - 2 ** b) * np.maximum(1, x)).max() <= 1e-7
