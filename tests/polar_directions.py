"""Matrices whose updates have few directions, as gradients of few examples are,
and how far a bf16 result of the orthogonalisation may be from the formula.

What the kernels keep of a bf16 result's steps: X as two halves, A and B as one
without their diagonals, and B X as (B - E) (upper half + lower half) of X with E,
the diagonal of B, in 32 bits; in the last two steps of matrices with more than 64
rows and columns the upper half alone. `held` takes the steps in 64 bits and rounds
there. With both halves every step is a product M X of the X that is held, so that
no direction comes in that X does not have but by 2^-23 of it. Of the upper half
alone, E times its rounding stays behind where B has no direction; a step more
multiplies that by the first coefficient.

BEFORE is what include/hkv_train.h says of results before their own rounding, in the
2-norm. The rounding is added from the steps of the values themselves: uniform, the
square of its norm is the sum of step^2 / 12. Over the 4000 elements and more that
these tests have, that sum is off by 2 %, and the product of both errors, which are
independent, by 2 / sqrt(4000) of their norms' product: 15 % covers both.
"""

import torch

import polar_reference as P

BEFORE = 1.7e-3


def most(steps):
    """A direction that X has by the halves' rounding alone, 2^-23 of it, grows by the
    first coefficient a step: 10 steps of it are 2.3e5 times as much. What the others
    are off by grows as well, by less than twice a step."""
    if steps <= 6:
        return BEFORE
    return BEFORE * 2 ** (steps - 6) + P.COEFFICIENTS[0] ** steps * 2.0 ** -23


def low(m, n, rank, kind, seed):
    """rank examples' X^T dY, in float32: of signed activations, of positive ones, of few that are not 0."""
    gen = torch.Generator().manual_seed(seed)
    x, dy = torch.randn(m, rank, generator=gen), torch.randn(rank, n, generator=gen)
    if kind == "positive":
        x = x.relu() + 1e-3
    if kind == "sparse":
        x = x * (torch.rand(m, rank, generator=gen) < 0.3)
        x[0] = 1.0
    return 1e-2 * (x @ dy)


def held(u, steps, narrow):
    x, flip = P.start(u, 1e-7)
    for k, (a, b, c) in enumerate(P.triples(steps, P.COEFFICIENTS)):
        hi, _, full = P.halves(x, True)
        g = hi @ hi.t()
        d = g.diagonal().clone()
        g = P.halves(g - torch.diag(d), False)[2]
        s = b * g + c * (g @ g + (d[:, None] + d[None]) * g)
        e = b * d + c * d * d + s.diagonal()
        s = P.halves(s - torch.diag(s.diagonal()), False)[2]
        x = (a + e)[:, None] * full + s @ (full if narrow or k < steps - 2 else hi)
    return x.t() if flip else x


def assert_rounded(got, want, steps, what):
    """got, bf16, is off from want by no more than BEFORE and its rounding."""
    got, want = got.double().cpu(), want.cpu()
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -120))) - 7)
    allowed = 1.15 * (float((step ** 2).sum()) / 12 + (most(steps) * float(want.norm())) ** 2)
    off = float((got - want).norm())
    assert off <= allowed ** 0.5, f"{what}: off by {off / float(want.norm()):.2e}, {allowed ** 0.5 / float(want.norm()):.2e} allowed"
