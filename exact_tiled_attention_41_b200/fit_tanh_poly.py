"""Fit the polynomials of the capped scores' tanh on the FMA pipe.

    python -m exact_tiled_attention_41_b200.fit_tanh_poly

tanh is odd, so tanh(x) = x p(x^2); p is fitted to tanh(sqrt(u)) / sqrt(u) on u in [0, R^2] with the smallest
maximum *relative* error (Remez exchange: equioscillation of p(u) sqrt(u) / tanh(sqrt(u)) - 1 at degree + 2 points).
Three ranges are used: degree 2 for |x| <= 1/4, degree 4 for |x| <= 1/2 and degree 6 for |x| <= 1.  The script prints the coefficients (highest
degree first, as Horner's rule in csrc/score.cuh uses them) and the worst relative error of the fp32 evaluation.
A CPU test re-runs the fit and compares it with the header.
"""

import numpy as np

RANGES = ((0.25, 2), (0.5, 4), (1.0, 6))


def _target(u):
    x = np.sqrt(np.maximum(u, 1e-12))
    return np.tanh(x) / x


def remez(limit, degree, iters=30):
    """Coefficients, lowest degree first, of the polynomial in u = x^2 on [0, limit^2]."""
    n, hi = degree + 2, limit * limit
    xs = hi / 2 - hi / 2 * np.cos(np.pi * np.arange(n) / (n - 1))
    grid = np.linspace(0.0, hi, 200001)
    f = _target(grid)
    for _ in range(iters):
        fx = _target(xs)
        m = np.vander(xs, degree + 1, increasing=True)
        m = np.hstack([m, ((-1.0) ** np.arange(n) * fx)[:, None]])
        c = np.linalg.solve(m, fx)[:-1]
        err = np.polyval(c[::-1], grid) / f - 1.0
        turn = np.flatnonzero((err[1:-1] - err[:-2]) * (err[2:] - err[1:-1]) <= 0) + 1
        picked = []
        for i in np.concatenate([[0], turn, [len(grid) - 1]]):
            if picked and np.sign(err[i]) == np.sign(err[picked[-1]]):
                if abs(err[i]) > abs(err[picked[-1]]):
                    picked[-1] = i
            else:
                picked.append(i)
        while len(picked) > n:
            picked.pop(0 if abs(err[picked[0]]) < abs(err[picked[-1]]) else -1)
        if len(picked) == n:
            xs = grid[picked]
    return c


def coefficients_f32(limit, degree):
    """The coefficients rounded to float32, highest degree first."""
    return [np.float32(a) for a in remez(limit, degree)[::-1]]


def fp32_error(limit, degree):
    """Worst relative error of the fp32 evaluation (separate roundings; fused ones are at least as accurate)."""
    x = np.linspace(1e-3, limit, 1_000_001).astype(np.float32)
    u = x * x
    c = coefficients_f32(limit, degree)
    p = np.full_like(u, c[0])
    for a in c[1:]:
        p = p * u + a
    return np.max(np.abs((p * x).astype(np.float64) / np.tanh(x.astype(np.float64)) - 1.0))


if __name__ == "__main__":
    for limit, degree in RANGES:
        print(f"|x| <= {limit}, degree {degree}: max relative error in fp32 {fp32_error(limit, degree):.3g}")
        print("  " + ", ".join(f"{a:.9g}f" for a in coefficients_f32(limit, degree)))
