"""Matrices whose rows would reach past any memory are refused: their extent is
more than 64 bits of bytes hold, so that no check of it against an allocation
could tell."""

import array

import pytest

import polar_reference as P
from test_training_abi import last

ADDRESS = 4096
FAR = dict(rows=1 << 24, cols=4, stride=1 << 40)  # 2^66 bytes of float32


@pytest.mark.parametrize("which", ["in", "out"])
def test_orthogonalize(which):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    strides = [FAR["stride"] if which == side else FAR["cols"] for side in ("in", "out")]
    item = array.array("Q", [ADDRESS, ADDRESS, FAR["rows"], FAR["cols"], *strides, 0, 0])
    c = array.array("d", list(P.COEFFICIENTS) * 5)
    st = T.load().hkv_orthogonalize(1, item.buffer_info()[0], 5, c.buffer_info()[0], 1e-7, None, 0, None)
    assert st == _native.HKV_EINVAL and f"{which}[0]" in last() and "past any memory" in last(), last()


@pytest.mark.parametrize("which", ["weight", "grad", "momentum"])
def test_muon(which):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    strides = [FAR["stride"] if which == side else FAR["cols"] for side in ("weight", "grad", "momentum")]
    item = T._MUON_MATRIX.pack(ADDRESS, ADDRESS, ADDRESS, FAR["rows"], FAR["cols"], *strides, 0, 0, 0.1, 1.0)
    c = array.array("d", list(P.COEFFICIENTS) * 5)
    st = T.load().hkv_muon_update(1, item, 0.9, 1, 0.0, 5, c.buffer_info()[0], 1e-7, None, 0, None)
    assert st == _native.HKV_EINVAL and f"{which}[0]" in last() and "past any memory" in last(), last()
