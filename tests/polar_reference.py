"""Orthogonalisation in 64 bits on the CPU, from its formula, and how far the
kernels may be from it.

The kernels hold X, A and B as halves: one (single) or the sum of two (split),
scaled by 2^12. `held` takes the same steps in 64 bits and rounds at the same
places, so that its distance from the formula is what these roundings cost for
the matrix at hand, whatever its spectrum. What it does not have is the rounding
of sums in 32 bits: a sum of q products is off by about sqrt(q) eps of its size,
which moves a step's X by that much relatively, and the result by kappa times as
much, kappa being measured on the formula with a random change of X in its first
and its last step. A rounding's random signs leave a factor of 2 between two such
errors of equal size; the tolerance takes 4 times the first and 8 times the second.
"""

import torch

import training_reference as R

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
UNIT = 4096.0


def triples(steps, coefficients):
    return list(coefficients) if isinstance(coefficients[0], (list, tuple)) else [coefficients] * steps


def start(u, eps):
    """X of the first step, its rows the shorter side, and whether it was transposed."""
    x = u / max(float(u.square().sum().sqrt()), eps)
    return (x.t(), True) if u.shape[0] > u.shape[1] else (x, False)


def polar(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7, first=None, last=None):
    """first, last: added to X before the first and the last step."""
    x, flip = start(u, eps)
    c = triples(steps, coefficients)
    for k, (a, b, d) in enumerate(c):
        if first is not None and k == 0:
            x = x + first
        if last is not None and k == len(c) - 1:
            x = x + last
        g = x @ x.t()
        x = a * x + (b * g + d * (g @ g)) @ x
    return x.t() if flip else x


def halves(x, split):
    """What the kernels hold of x: the upper half of every number, and both where split."""
    hi = (x * UNIT).half().double() / UNIT
    lo = ((x - hi) * UNIT).half().double() / UNIT
    return hi, lo, hi + lo if split else hi


def held(u, steps, coefficients, eps, split):
    x, flip = start(u, eps)
    for a, b, c in triples(steps, coefficients):
        hi, lo, x1 = halves(x, split)
        g = x1 @ x1.t()
        d = g.diagonal().clone()
        g = halves(g - torch.diag(d), split)[2]
        s = b * g + c * (g @ g + (d[:, None] + d[None]) * g)
        e = b * d + c * d * d + s.diagonal()
        s = halves(s - torch.diag(s.diagonal()), split)[2]
        x = (a + e)[:, None] * (hi + lo) + s @ x1
    return x.t() if flip else x


def tolerance(u, steps, coefficients, eps, split):
    """The formula's result, and how far (2-norm) the kernels' may be before their last rounding."""
    want = polar(u, steps, coefficients, eps)
    model = float((held(u, steps, coefficients, eps, split) - want).norm())
    x, _ = start(u, eps)
    gen = torch.Generator().manual_seed(1)
    noise = torch.randn(x.shape, generator=gen, dtype=torch.float64)
    noise /= noise.norm()
    h = 1e-6
    moved = 0.0
    size = float(x.norm())
    for kw, n in (({"first": h * size * noise}, size), ({"last": h * float(want.norm()) * noise}, float(want.norm()))):
        moved = max(moved, float((polar(u, steps, coefficients, eps, **kw) - want).norm()) / h)
    # a change of X's length, which all sums of a step share, moves all singular values alike
    moved = max(moved, float((polar(u * (1 + h), steps, coefficients, 1e-300, first=h * x) - want).norm()) / h)
    return want, 4 * model + 8 * moved * max(u.shape) ** 0.5 * R.EPS


def assert_polar(got, u, steps=5, coefficients=COEFFICIENTS, eps=1e-7, what=""):
    want, tol = tolerance(u, steps, coefficients, eps, got.dtype != torch.bfloat16)
    assert_close(got, want, tol, what)


def assert_close(got, want, tol, what):
    """Within tol in the 2-norm and, element by element, 10 times the root mean
    square that this leaves; each after half a step of got's type."""
    half = R.half_step(got.dtype)
    off = (R.f64(got) - want).abs()
    assert bool(off.isfinite().all()), f"{what}: not finite"
    rms = tol / max(1, want.numel()) ** 0.5
    step = half * (want.abs() + 10 * rms) + R.TINY[got.dtype]
    assert float(off.norm()) <= tol + float(step.norm()), f"{what}: off by {float(off.norm()):.3e}, {tol:.3e} allowed"
    worst = (off - step).max()
    assert float(worst) <= 10 * rms, f"{what}: an element off by {float(worst):.3e}, {10 * rms:.3e} allowed"
