"""bf16 results of matrices of few directions, against the bound that the header
states: every kernel, one block of columns and many, tiles of every size, and the
momentum update. The model's own bound (polar_reference.tolerance) grows with what
the kernels lose; this one does not."""

import pytest
import torch

import polar_directions as D
import polar_reference as P
from conftest import gpu_available
from test_gpu_orthogonalize import dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

RANKS = (1, 4, 16, 32)
KINDS = ("signed", "positive", "sparse")


@pytest.mark.parametrize("steps", [5, 6, 10])
@pytest.mark.parametrize("shape", [(64, 64), (40, 100), (64, 256), (20, 300), (2500, 60), (128, 512), (300, 200),
                                   (200, 9000)])
def test_few_directions(shape, steps):
    import hash_table_cache_amd as H

    which = [(rank, kind) for rank in RANKS for kind in KINDS if rank < min(shape)]
    us = [D.low(*shape, rank, kind, rank).to(dev()) for rank, kind in which]
    outs = [torch.empty(shape, dtype=torch.bfloat16, device=dev()) for _ in us]
    for (rank, kind), u, o in zip(which, us, H.orthogonalize(us, steps=steps, out=outs)):
        D.assert_rounded(o, P.polar(u.double(), steps), steps, f"{kind} {rank} of {shape}")


@pytest.mark.parametrize("shape,count", [((300, 500), 12), ((800, 1600), 6), ((1100, 2300), 6), ((1000, 2000), 8)])
def test_tiles(shape, count):
    """Tiles of 64, 128 and 256."""
    import hash_table_cache_amd as H

    us = [D.low(*shape, (1, 8, 32, 100)[i % 4], KINDS[i % 3], i).to(dev()) for i in range(count)]
    outs = [torch.empty(shape, dtype=torch.bfloat16, device=dev()) for _ in us]
    for i, (u, o) in enumerate(zip(us, H.orthogonalize(us, steps=6, out=outs))):
        D.assert_rounded(o, P.polar(u.double(), 6), 6, f"{i} of {shape}")


@pytest.mark.parametrize("nesterov", [True, False])
def test_update_of_bf16_weights(nesterov):
    """Gradients and momenta in float32, weights of 0, so that they are the result itself."""
    import hash_table_cache_amd as H

    shapes = [(64, 64), (64, 256), (256, 40), (128, 512), (300, 200)]
    g = [D.low(*s, rank, kind, rank).to(dev()) for s in shapes for rank in RANKS for kind in KINDS]
    w = [torch.zeros(x.shape, dtype=torch.bfloat16, device=dev()) for x in g]
    m = [torch.zeros_like(x) for x in g]
    H.muon_update(w, g, m, -1.0, momentum=0.5, nesterov=nesterov, scale=None)
    for x, y, z in zip(g, w, m):
        kept = z.double()  # 0.5 g, exactly
        u = 0.5 * x.double() + 0.5 * kept if nesterov else kept
        D.assert_rounded(y, P.polar(u), 5, f"{tuple(x.shape)}")
