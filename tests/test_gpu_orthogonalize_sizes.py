"""Orthogonalisation where calls change their way: narrow matrices of one block
of columns and of many, tiles of A shared along long rows, tiles of each size, and
lists longer than a launch's arguments or a workspace take.

Narrow ones are held to polar_reference's tolerance. Large ones are compared with
their own steps in 64 bits on the GPU, by 2-norm: a bf16 result is off by its
rounding, at most 2^-9 of a number on the average, and by less than that before it
(together under 4.6e-3); a float32 result by sums of up to 2^16 terms, each term
off by 2^-22 with a random sign and each sum by 2^-24 for the blocks of 64 that it
grows by (under 1e-5).
"""

import pytest
import torch

import polar_reference as P
import training_reference as R
from conftest import gpu_available
from test_gpu_orthogonalize import dev, make, update

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BOTH = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("p", [1, 16, 17, 32, 33, 49, 64])
def test_narrow(p, dtype):
    """One block of 256 columns, several, and so many that their parts are added by a launch of their own."""
    import hash_table_cache_amd as H

    us = [make(*((p, q) if i % 2 else (q, p)), dtype, p + i, ("full", "low", "decay")[i % 3], i % 4)
          for i, q in enumerate((256, 257, 1000, 2048, 2049, 8200, 20011))]
    for got, u in zip(H.orthogonalize(us), us):
        P.assert_polar(got, R.f64(u), what=f"{tuple(u.shape)}")
        alone = H.orthogonalize([u])[0]
        assert torch.equal(alone, got)


@pytest.mark.parametrize("count", [1, 2, 15, 16, 17, 40])
def test_lists_longer_than_arguments(count):
    """Small matrices of one block, of several, and of more than 64 rows, as many as fit and more."""
    import hash_table_cache_amd as H

    for m, n in ((20, 30), (40, 300), (70, 80)):
        for dtype in BOTH:
            us = [make(m, n, dtype, i, ("full", "low")[i % 2], i % 3) for i in range(count)]
            for i, (got, u) in enumerate(zip(H.orthogonalize(us), us)):
                P.assert_polar(got, R.f64(u), what=f"{i} of {count}")


def compare(us, what):
    import hash_table_cache_amd as H

    got = H.orthogonalize(us)
    for o, u in zip(got, us):
        want = P.polar(u.double())
        rel = float((o.double() - want).norm() / want.norm())
        assert rel < (4.6e-3 if o.dtype == torch.bfloat16 else 1e-5), (what, tuple(u.shape), rel)
    return got


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("shapes", [
    [(65, 4000)], [(100, 3000), (3001, 99), (70, 65)], [(200, 60000)], [(60001, 70)],  # A's tiles shared along rows
    [(50, 66001)], [(66000, 64), (20, 70000)],  # narrow, but longer than their own kernels take
    [(1024, 1024)] * 8, [(1024, 2048)] * 4, [(2048, 1000)] * 4, [(500, 1300)] * 12,  # tiles of 64 and 128
    [(1024, 2048)] * 8, [(4096, 4096)], [(2300, 2100), (4097, 4095), (70, 5000)],  # of 256
])
def test_ways(shapes, dtype):
    gen = torch.Generator(device=dev()).manual_seed(2)
    us = [(torch.randn(s, device=dev(), generator=gen) * 0.01).to(dtype) for s in shapes]
    compare(us, shapes[0])


def test_more_than_a_workspace_takes():
    """Their scratch passes 4 GiB: two groups, one after the other in the same memory."""
    import hash_table_cache_amd as H

    gen = torch.Generator(device=dev()).manual_seed(3)
    us = [torch.randn(2048, 4000, device=dev(), generator=gen).to(torch.bfloat16) for _ in range(44)]
    got = compare(us, "many")
    for i in (0, 20, 43):  # as alone, within the rounding of tiles of another size
        alone = H.orthogonalize([us[i]])[0].double()
        assert float((alone - got[i].double()).norm() / alone.norm()) < 4.6e-3


def test_the_same_bits_again():
    import hash_table_cache_amd as H

    for shape, n in (((50, 3000), 3), ((200, 9000), 2), ((1024, 2048), 4)):
        for dtype in BOTH:
            us = [make(*shape, dtype, i) for i in range(n)]
            for a, b in zip(H.orthogonalize(us), H.orthogonalize(us)):
                assert torch.equal(a, b)


def test_rows_next_to_others():
    """Of results in wider rows, tiles of 128 and 256 write their own columns only, whatever the alignment."""
    import hash_table_cache_amd as H

    for shape, n in (((1030, 1025), 8), ((1030, 2049), 8)):
        us = [make(*shape, torch.bfloat16, i) for i in range(n)]
        plain = H.orthogonalize(us)
        wide = [torch.full((shape[0] + 1, shape[1] + 9), 7.0, dtype=torch.bfloat16, device=dev()) for _ in us]
        outs = [w[:shape[0], 1 + i % 8:1 + i % 8 + shape[1]] for i, w in enumerate(wide)]
        H.orthogonalize(us, out=outs)
        for i, (w, o, p) in enumerate(zip(wide, outs, plain)):
            assert torch.equal(o, p)
            assert bool((w[shape[0]:] == 7).all())
            assert bool((w[:, :1 + i % 8] == 7).all()) and bool((w[:, 1 + i % 8 + shape[1]:] == 7).all())


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", BOTH)
def test_muon_of_tall_and_long(nesterov, dtype):
    """Narrow weights of one block and of several, and larger ones, with and without the look ahead."""
    import hash_table_cache_amd as H

    shapes = [(300, 20), (700, 33), (1500, 8), (30, 700), (256, 64), (64, 2000), (400, 90), (90, 5000)]
    w = [(100 * make(a, b, torch.float32, i, pad=i % 3)).to(dtype) for i, (a, b) in enumerate(shapes)]
    g = [make(a, b, dtype, 20 + i, ("full", "low", "decay")[i % 3], (i + 1) % 3) for i, (a, b) in enumerate(shapes)]
    m = [make(a, b, torch.float32, 40 + i, pad=(i + 2) % 3) for i, (a, b) in enumerate(shapes)]
    want = [update(a, b, c, 0.2, 1.0, 0.8, nesterov, 0.05, 5, P.COEFFICIENTS, 1e-7) for a, b, c in zip(w, g, m)]
    H.muon_update(w, g, m, 0.2, momentum=0.8, nesterov=nesterov, weight_decay=0.05, scale=None)
    for i, (moved, weight, tol) in enumerate(want):
        R.assert_near(m[i], moved, moved.abs() * R.EPS + R.TINY[torch.float32], f"momentum {i}")
        P.assert_close(w[i], weight, tol, f"weight {i}")
