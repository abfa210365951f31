"""Orthogonalisation's entry points refuse bad arguments before touching a GPU,
and the reference of its tests is what it says."""

import array

import pytest
import torch

import polar_reference as P
from test_training_abi import last

ADDRESS = 4096


def matrices(rows=8, cols=9, in_stride=9, out_stride=9, in_dtype=0, out_dtype=0):
    return array.array("Q", [ADDRESS, ADDRESS, rows, cols, in_stride, out_stride, in_dtype, out_dtype])


def run(list_=None, n=1, steps=5, c=P.COEFFICIENTS, eps=1e-7):
    from hash_table_cache_amd import training as T

    list_ = matrices() if list_ is None else list_
    flat = array.array("d", list(c) * max(1, min(steps, 100)))
    return T.load().hkv_orthogonalize(n, list_.buffer_info()[0], steps, flat.buffer_info()[0], eps, None, 0, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(n=1 << 20), "matrices"), (dict(steps=0), "steps"), (dict(steps=65), "steps"), (dict(eps=0.0), "eps"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(c=(float("nan"), 0.0, 0.0)), "finite"), (dict(c=(3.95, 0.0, 0.0)), "range"),
    (dict(c=(1.5, -16.0, 0.0)), "range"), (dict(c=(2.0, 0.0, 0.0)), "range"),
    (dict(list_=matrices(rows=1 << 25)), "2\\^24"), (dict(list_=matrices(rows=1 << 16, cols=1 << 16, in_stride=1 << 16)), "2\\^15"),
    (dict(list_=matrices(in_stride=8)), "stride"), (dict(list_=matrices(out_stride=1 << 41)), "stride"),
    (dict(list_=matrices(in_dtype=3)), "dtype"), (dict(list_=matrices(out_dtype=1 << 32)), "dtype"),
    (dict(list_=matrices()), "in\\[0\\]"),
])
def test_orthogonalize_refuses(kw, needle):
    import re

    from hash_table_cache_amd import _native

    assert run(**kw) == _native.HKV_EINVAL and re.search(needle, last()), last()


@pytest.mark.parametrize("c,steps", [(P.COEFFICIENTS, 64), ((1.5, -0.5, 0.0), 64), ((15 / 8, -10 / 8, 3 / 8), 64),
                                     ((8.2872, -23.5959, 17.3004), 1)])
def test_usual_coefficients_are_taken(c, steps):
    from hash_table_cache_amd import _native

    assert run(matrices(rows=0), c=c, steps=steps) == _native.HKV_OK


@pytest.mark.parametrize("kw,needle", [
    (dict(momentum=1.0), "momentum"), (dict(momentum=-0.5), "momentum"), (dict(momentum=float("nan")), "momentum"),
    (dict(nesterov=2), "nesterov"), (dict(decay=float("inf")), "weight_decay"), (dict(steps=0), "steps"),
    (dict(eps=0.0), "eps"), (dict(lr=float("nan")), "lr"), (dict(scale=float("inf")), "scale"), (dict(), "weight"),
])
def test_muon_refuses(kw, needle):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    a = dict(momentum=0.9, nesterov=1, decay=0.0, steps=5, eps=1e-7, lr=0.1, scale=1.0) | kw
    item = T._MUON_MATRIX.pack(ADDRESS, ADDRESS, ADDRESS, 8, 9, 9, 9, 9, 0, 0, a["lr"], a["scale"])
    c = array.array("d", list(P.COEFFICIENTS) * 5)
    st = T.load().hkv_muon_update(1, item, a["momentum"], a["nesterov"], a["decay"], a["steps"], c.buffer_info()[0],
                                  a["eps"], None, 0, None)
    assert st == _native.HKV_EINVAL and needle in last(), last()


def test_null_lists_and_empty_ones():
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    values = array.array("d", list(P.COEFFICIENTS) * 5)
    c = values.buffer_info()[0]
    one = matrices()
    L = T.load()
    assert L.hkv_orthogonalize(0, None, 5, c, 1e-7, None, 0, None) == _native.HKV_OK
    assert L.hkv_orthogonalize(1, None, 5, c, 1e-7, None, 0, None) == _native.HKV_EINVAL and "NULL" in last()
    assert L.hkv_orthogonalize(1, one.buffer_info()[0], 5, None, 1e-7, None, 0, None) == _native.HKV_EINVAL
    assert "coefficients" in last()
    assert L.hkv_muon_update(1, None, 0.9, 1, 0.0, 5, c, 1e-7, None, 0, None) == _native.HKV_EINVAL and "NULL" in last()


def test_workspace():
    from hash_table_cache_amd import training as T

    def need(shapes, kind):
        return T._polar_workspace_bytes(tuple(shapes), bytes([kind]) * len(shapes))

    assert need([(0, 5)], 0) == 0
    assert need([(500, 400)], 0) > need([(500, 400)], 1) > need([(200, 400)], 1) > 0
    assert need([(500, 400)] * 3, 1) > need([(500, 400)], 1)
    # long lists are worked on in groups: the workspace does not grow without end
    assert need([(4096, 4096)] * 400, 0) < 6 << 30


def test_python_checks_come_first():
    import hash_table_cache_amd as H

    u = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        H.orthogonalize([u])
    with pytest.raises(ValueError, match="at least one"):
        H.orthogonalize([])
    with pytest.raises(ValueError, match="GPU"):
        H.muon_update([u], [u], [u], 0.1)
    with pytest.raises(ValueError, match="at least one"):
        H.muon_update([], [], [], 0.1)
    with pytest.raises(ValueError, match="gradients"):
        H.muon_update([u], [], [u], 0.1)


def test_reference():
    """The 64-bit steps reach U V^T; what the kernels hold costs as much as is claimed."""
    gen = torch.Generator().manual_seed(0)
    u = torch.randn(40, 60, generator=gen, dtype=torch.float64)
    a, _, b = torch.linalg.svd(u, full_matrices=False)
    assert float((P.polar(u, 30, (15 / 8, -10 / 8, 3 / 8)) - a @ b).abs().max()) < 1e-12
    assert torch.allclose(P.polar(u.t()).t(), P.polar(u), rtol=0, atol=1e-12)
    for shape, rank in (((64, 64), 0), ((200, 300), 0), ((256, 256), 8)):
        u = torch.randn(shape, generator=gen, dtype=torch.float64)
        if rank:
            u = torch.randn(shape[0], rank, generator=gen, dtype=torch.float64) @ torch.randn(rank, shape[1], generator=gen, dtype=torch.float64)
        want = P.polar(u)
        # noise of 2^-24 of X in directions that have no singular value grows 3.4445^5 times, the 8 others 2.5 times
        for split, most in ((False, 1.3e-3), (True, 1.2e-5 if rank else 2e-6)):
            rel = float((P.held(u, 5, P.COEFFICIENTS, 1e-7, split) - want).norm() / want.norm())
            assert rel < most, (shape, split, rel)
