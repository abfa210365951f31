"""The token statistics' entry points refuse bad arguments before touching a GPU."""

import pytest
import torch

from test_training_abi import BAD_LOGITS, P, last, logits_args


@pytest.mark.parametrize("kw,needle", BAD_LOGITS)
def test_logits_are_refused(kw, needle):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    L = T.load()
    a = logits_args(**kw)
    assert L.hkv_token_stats(*a, 4, P, P, P, P, P, P, 1 << 20, None) == _native.HKV_EINVAL and needle in last()
    assert L.hkv_token_stats_backward(*a, P, P, P, P, P, 1 << 30, None) == _native.HKV_EINVAL and needle in last()


def test_arguments_are_refused():
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    L = T.load()
    assert L.hkv_token_stats(*logits_args(), 65, P, P, P, P, P, P, 1 << 20, None) == _native.HKV_EINVAL
    assert "k = 65" in last()
    assert L.hkv_token_stats_backward(*logits_args(), P, P, None, None, P, 8, None) == _native.HKV_EINVAL
    assert "grad_logp and grad_entropy" in last()
    assert L.hkv_token_stats_backward(*logits_args(), P, P, P, P, None, 8, None) == _native.HKV_EINVAL
    assert "grad_out" in last()
    assert L.hkv_token_stats_backward(*logits_args(), P, P, P, P, P, 7, None) == _native.HKV_EINVAL
    assert "grad_stride" in last()


def test_host_memory_is_refused():
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    host, y = torch.zeros(64), torch.zeros(4, dtype=torch.int64)
    st = T.load().hkv_token_stats(4, 8, 0, host.data_ptr(), 8, y.data_ptr(), 1.0, 2, host.data_ptr(), None,
                                  host.data_ptr(), host.data_ptr(), y.data_ptr(), None, 0, None)
    assert st == _native.HKV_EINVAL and "logits" in last()


def test_workspace():
    from hash_table_cache_amd import training as T

    w = T.load().hkv_token_stats_workspace_bytes
    assert w(100000, 1 << 17, 1, 64) == 0  # rows enough for a workgroup each
    assert w(0, 1 << 17, 1, 5) == 0
    assert w(1, 100, 0, 5) == 0  # short
    assert w(4, 1 << 17, 1, 5) > w(1, 1 << 17, 1, 5) > w(1, 1 << 17, 1, 0) > 0
    assert w(1 << 31, 1 << 17, 1, 5) == 0


def test_python_checks_come_first():
    import hash_table_cache_amd as H

    x, y = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        H.token_stats(x, y, 3)
    with pytest.raises(TypeError, match="float64"):
        H.token_stats(x.double(), y)
    with pytest.raises(ValueError, match="GPU"):
        H.token_stats_backward(x, y, x[:, 0], x[:, 0], x[:, 0])
