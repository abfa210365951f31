"""What bf16 results of the orthogonalisation hold costs no more than is claimed,
whatever the number of directions."""

import pytest

import polar_directions as D
import polar_reference as P


@pytest.mark.parametrize("kind", ["signed", "positive", "sparse"])
@pytest.mark.parametrize("shape", [(64, 64), (40, 100), (64, 256), (128, 512), (300, 200)])
def test_few_directions(shape, kind):
    for rank in (1, 4, 16, 32):
        for steps in (1, 2, 3, 5, 6, 10):
            u = D.low(*shape, rank, kind, rank).double()
            want = P.polar(u, steps)
            off = float((D.held(u, steps, min(shape) <= 64) - want).norm() / want.norm())
            assert off < D.most(steps), (shape, rank, steps, off)
