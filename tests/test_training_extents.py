"""Extents of [rows][vocab] arrays that pass 64 bits are refused: rows times a
stride that wraps around would look like a small array that holds the call. No
kernels run."""

import ctypes

import pytest

# stands for a device address; the refusals come before any look at it
P = ctypes.c_void_p(4096)


def calls(rows, vocab, dtype, stride, grad_stride):
    from hash_table_cache_amd import training as T

    L = T.load()
    a = [rows, vocab, dtype, P, stride, P, 1.0]
    yield "logprobs", L.hkv_token_logprobs(*a, P, P, P, 1 << 50, None)
    yield "backward", L.hkv_token_logprobs_backward(*a, P, P, P, grad_stride, None)
    yield "preference", L.hkv_preference_loss(*a, 1, P, P, .1, 0., 1., P, P, P, P, P, grad_stride, P, 1 << 50, None)
    yield "policy", L.hkv_policy_loss(*a, P, P, P, P, .2, .2, 0., 1., P, P, P, P, P, grad_stride, P, 1 << 50, None)


# (rows - 1) * stride: 2^64 elements, 2^62 of 4 bytes, 2^63 of 2 bytes, the most that rows and strides could be
@pytest.mark.parametrize("rows,stride,dtype", [((1 << 24) + 1, 1 << 40, 0), ((1 << 22) + 1, 1 << 40, 0),
                                               ((1 << 23) + 1, 1 << 40, 1), ((1 << 31) - 1, 1 << 40, 2),
                                               ((1 << 31) - 1, (1 << 33) + 8, 0)])
def test_extents_past_64_bits(rows, stride, dtype):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    for name, status in calls(rows, 8, dtype, stride, stride):
        assert status == _native.HKV_EINVAL, name
        assert "logits_stride" in T.load().hkv_train_last_error().decode(), name
    for name, status in calls(rows, 8, dtype, 8, stride):
        assert status == _native.HKV_EINVAL, name
        if name != "logprobs":
            assert "grad_stride" in T.load().hkv_train_last_error().decode(), name


def test_one_row_may_have_any_stride():
    """The stride of a single row is not used: the next check is the one that speaks."""
    from hash_table_cache_amd import training as T

    for name, _ in calls(1, 8, 0, 1 << 40, 1 << 40):
        assert "stride" not in T.load().hkv_train_last_error().decode(), name
