"""Fits the polynomial of gated_ff.cuh's gelu_pair: log2 of the normal tail.

    q(x) = erfc(x / sqrt 2) / 2 = 2^P(-x),   x in [0, 5.6], P of degree 7

(the kernel uses P down to -8: it falls on, and x q stays below 1e-7).

Method: weighted minimax by Lawson's iteration (least squares whose weights are
multiplied by the errors until these are level), in a Chebyshev basis; the
weight ln 2 q max(1, x) turns an error of P into the errors of q and x q.
Prints the coefficients rounded to fp32, as Horner's rule in m = -x takes them.
"""
import numpy as np
from numpy.polynomial import chebyshev, polynomial
from scipy.special import erfc, log_ndtr

BOUND, DEGREE = 5.6, 7


def fit():
    x = np.linspace(0, BOUND, 4001)
    target = log_ndtr(-x) / np.log(2)
    weight = np.log(2) * 0.5 * erfc(x / np.sqrt(2)) * np.maximum(1, x)
    basis = chebyshev.chebvander(2 * x / BOUND - 1, DEGREE)
    lam, best = np.ones_like(x) / x.size, (np.inf, None)
    for _ in range(3000):
        w = np.sqrt(lam) * weight
        c = np.linalg.lstsq(basis * w[:, None], target * w, rcond=None)[0]
        err = np.abs(basis @ c - target) * weight
        if err.max() < best[0]:
            best = (err.max(), c)
        lam = lam * (err + 1e-300)
        lam /= lam.sum()
    p = np.zeros(1)
    for a in chebyshev.cheb2poly(best[1])[::-1]:
        p = polynomial.polyadd(polynomial.polymul(p, [-1.0, -2 / BOUND]), [a])   # x = -m
    return best[0], p.astype(np.float32)


if __name__ == "__main__":
    err, p = fit()
    print(f"largest weighted error {err:.2e}")
    for k, v in enumerate(p):
        print(f"kTail{k} = {float(v)!r}")
