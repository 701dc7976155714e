"""Fit the polynomials of the rotary tables' sines and cosines.

    python -m exact_tiled_attention_41_b200.fit_trig_poly

The tables' angles are reduced to y in [-pi/4, pi/4] as integers (csrc/rotary.cu).  There sin(y) = y p(y^2) and
cos(y) = q(y^2), with p of degree 3 and q of degree 4 fitted for the smallest maximum relative error (Remez exchange, as
in fit_tanh_poly.py).  The script prints the coefficients (highest degree first, as Horner's rule uses them) and the
worst absolute error of the fp32 evaluation; a CPU test re-runs the fit and compares it with the source.
"""

import numpy as np

HI = (np.pi / 4) ** 2


def _sin(u):
    y = np.sqrt(np.maximum(u, 1e-16))
    return np.sin(y) / y


def _cos(u):
    return np.cos(np.sqrt(u))


FITS = {"sin": (_sin, 3), "cos": (_cos, 4)}


def remez(name, iters=30):
    """Coefficients, lowest degree first, in u = y^2 on [0, (pi/4)^2]."""
    target, degree = FITS[name]
    n = degree + 2
    xs = HI / 2 - HI / 2 * np.cos(np.pi * np.arange(n) / (n - 1))
    grid = np.linspace(0.0, HI, 200001)
    f = target(grid)
    for _ in range(iters):
        fx = target(xs)
        m = np.hstack([np.vander(xs, degree + 1, increasing=True), ((-1.0) ** np.arange(n) * fx)[:, None]])
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
        if len(picked) != n:
            break        # the error is down at rounding: the last solution stands
        xs = grid[picked]
    return c


def coefficients_f32(name):
    """The coefficients rounded to float32, highest degree first."""
    return [np.float32(a) for a in remez(name)[::-1]]


def fp32_error(name):
    """Worst absolute error over the reduced range, evaluated in fp32 with separate roundings."""
    y = np.linspace(-np.pi / 4, np.pi / 4, 1_000_001).astype(np.float32)
    u = y * y
    c = coefficients_f32(name)
    p = np.full_like(u, c[0])
    for a in c[1:]:
        p = p * u + a
    got = (p * y if name == "sin" else p).astype(np.float64)
    return np.max(np.abs(got - getattr(np, name)(y.astype(np.float64))))


if __name__ == "__main__":
    for name in FITS:
        print(f"{name}: max absolute error in fp32 {fp32_error(name):.3g}")
        print("  " + ", ".join(f"{a:.9g}f" for a in coefficients_f32(name)))
