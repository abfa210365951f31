"""Lists in which large and small matrices get tiles of different sizes, in any
order: every result as its own steps in 64 bits, and the same bits again."""

import pytest
import torch

import polar_reference as P
from conftest import gpu_available
from test_gpu_orthogonalize import dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shapes", [
    [(70, 70)] * 256, [(128, 129)] * 260,  # as many as large tiles would be taken for
    [(70, 70)] * 20 + [(4096, 4096)] + [(300, 500)] * 3 + [(60, 70000), (20, 30)],  # a large one, small ones apart
    [(1100, 1100)] * 11, [(768, 2048)] * 11,  # tiles of 256 would be a round and a little
    [(192, 4096), (4096, 200)] * 4 + [(1024, 2048)] * 8,
    [(1019, 2039), (2041, 1009)] * 4,  # tiles of 256 that end past the matrix
])
def test_mixed(shapes, dtype):
    import hash_table_cache_amd as H

    gen = torch.Generator(device=dev()).manual_seed(4)
    us = [(torch.randn(s, device=dev(), generator=gen) * 0.01).to(dtype) for s in shapes]
    got = H.orthogonalize(us)
    for i in range(0, len(us), 1 if len(us) < 50 else 37):
        want = P.polar(us[i].double())
        rel = float((got[i].double() - want).norm() / want.norm())
        # as in test_gpu_orthogonalize_sizes: bf16 its rounding and less before it, float32 sums of up to 2^17 terms
        assert rel < (4.6e-3 if dtype == torch.bfloat16 else 1e-5), (i, shapes[i], rel)
    for a, b in zip(got, H.orthogonalize(us)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_next_to_others(dtype):
    """Tiles of 256 write their own rows and columns only, whatever the alignment; so does the update."""
    import hash_table_cache_amd as H

    gen = torch.Generator(device=dev()).manual_seed(5)
    shapes = [(1019, 2039), (2041, 1009)] * 4
    us = [(torch.randn(s, device=dev(), generator=gen) * 0.01).to(dtype) for s in shapes]
    plain = H.orthogonalize(us)
    wide = [torch.full((m + 1, n + 9), 7.0, dtype=dtype, device=dev()) for m, n in shapes]
    outs = [w[:m, 1 + i % 8:1 + i % 8 + n] for i, (w, (m, n)) in enumerate(zip(wide, shapes))]
    H.orthogonalize(us, out=outs)
    momenta = [torch.zeros(s, device=dev()) for s in shapes]
    for once in range(2):
        for i, (w, o, p) in enumerate(zip(wide, outs, plain)):
            if not once:
                assert torch.equal(o, p)
            m, n = o.shape
            assert bool((w[m:] == 7).all())
            assert bool((w[:, :1 + i % 8] == 7).all()) and bool((w[:, 1 + i % 8 + n:] == 7).all())
        H.muon_update(outs, us, momenta, 0.1)
