"""Fits the upper tail of the normal distribution used by the gelu of
linear_gemm.hpp and its derivative.

Q(x) = erfc(x / sqrt 2) / 2 for x >= 0 is written e^{-x^2/2} P(u), u = 1 / (1 + 0.3 x),
with P a polynomial of degree 6 that minimises the relative error on [0, 14.5] (past it
Q is below the smallest bfloat16 subnormal): weighted least squares on Chebyshev-spaced
u, reweighted towards the minimax solution.  The target is scipy.special.erfcx.
Relative error of the fit: 1.9e-6, far below the 2^-9 and 2^-12 of the 16-bit outputs;
degree 8 (fit_erfc.py) costs two more multiply-adds an element, and the activations'
arithmetic is what the epilogues of short products spend their time on.

Run: python fit_normal_tail.py   (prints the coefficients, lowest degree first)
"""
import numpy as np
import scipy.special


def fit(deg: int = 6, a: float = 0.3, xmax: float = 14.5, n: int = 6000, rounds: int = 300):
    theta = (np.arange(n) + 0.5) / n * np.pi
    umin = 1 / (1 + a * xmax)
    u = umin + (1 - umin) * (0.5 - 0.5 * np.cos(theta))
    target = 0.5 * scipy.special.erfcx((1 / u - 1) / a / np.sqrt(2))
    rel = np.vander(u, deg + 1, increasing=True) / target[:, None]
    w = np.ones(n)
    for _ in range(rounds):
        s = np.sqrt(w)
        c = np.linalg.lstsq(rel * s[:, None], s, rcond=None)[0]
        err = np.abs(rel @ c - 1)
        w *= err + 1e-16
        w /= w.sum()
    return c, float(err.max())


if __name__ == "__main__":
    coeffs, max_rel = fit()
    print(f"max relative error of the fit: {max_rel:.3e}")
    print(", ".join(f"{float(np.float32(x)):.9e}f" for x in coeffs))
