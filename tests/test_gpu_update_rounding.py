"""Weights are rounded once to their type: a gradient of zeros leaves keep * w,
whose only rounding beside it is that of a product in 64 bits."""

import numpy as np
import pytest
import torch

from conftest import gpu_available
from test_gpu_orthogonalize import dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DIGITS = {torch.float32: 24, torch.bfloat16: 8, torch.float16: 11}
LOWEST = {torch.float32: -149, torch.bfloat16: -133, torch.float16: -24}  # exponent of the smallest step
# one block of columns, several, tiles of 64, of 256, both orientations
LISTS = [[(30, 40)], [(700, 50)], [(200, 300), (300, 200)], [(1019, 2039), (2041, 1009)] * 4]


def once(v, dtype):
    """v, in 64 bits, rounded to dtype: the nearest, of two the even one."""
    v = v.cpu().numpy()
    step = np.ldexp(1.0, np.maximum(np.frexp(v)[1] - DIGITS[dtype], LOWEST[dtype]))
    return torch.from_numpy(np.rint(v / step) * step)


@pytest.mark.parametrize("dtype", DIGITS)
@pytest.mark.parametrize("shapes", LISTS)
def test_weights(shapes, dtype):
    import hash_table_cache_amd as H

    gen = torch.Generator(device=dev()).manual_seed(1)
    middle = 2.0 ** -DIGITS[dtype]  # between 1 and the next number
    for decay in (-(middle + 2.0 ** -30), -(middle - 2.0 ** -30), -middle, 0.1, 1 / 3):
        w = [torch.randn(s, device=dev(), generator=gen).to(dtype) for s in shapes]
        for x in w:
            x[:, ::2] = 1.0
            x[1::2, ::2] = -1.0
            x[0, 1:9] = torch.tensor([0.0, -0.0, 1e-7, -3e-5, 6e-8, 1e-40, 3e4, 250.0], device=dev()).to(dtype)
        g = [torch.zeros_like(x) for x in w]
        want = [once((1.0 - decay) * x.double(), dtype) for x in w]
        H.muon_update(w, g, [torch.zeros(s, device=dev()) for s in shapes], 1.0, weight_decay=decay, scale=None)
        for x, y in zip(w, want):
            assert torch.equal(x.double().cpu(), y), decay
