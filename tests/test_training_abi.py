"""The training operators' library: it loads, exports what include/hkv_train.h
declares, and refuses bad arguments before touching a GPU. No kernels run."""

import ctypes
import pathlib
import re
import subprocess

import pytest
import torch

from conftest import ROOT

HEADER = pathlib.Path(ROOT) / "include" / "hkv_train.h"


def declared():
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\**(hkv_\w+)\s*\(", text, flags=re.M)))


def test_header_and_exports():
    from hash_table_cache_amd import training as T

    assert declared() == sorted(T.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", str(T.LIB_PATH)], check=True, capture_output=True,
                         text=True).stdout
    assert {l.split()[-1] for l in out.splitlines() if " T " in l and "hkv" in l} == set(declared())
    for name in declared():
        assert getattr(T.load(), name) is not None


def test_kernels_hold_no_packed_fp32():
    from hash_table_cache_amd import build as hb

    out = subprocess.run([hb.hipcc(), *hb.compile_flags(), "--offload-device-only", "-S", "-x", "hip",
                          str(hb.TRAIN_SOURCES[0]), "-o", "-"], capture_output=True, text=True, check=True)
    assert "gfx950" in out.stdout
    for op in ("add", "mul", "fma"):
        assert "v_pk_" + op + "_f32" not in out.stdout
    assert "scratch_store" not in out.stdout  # rows stay in registers


def test_workspace_grows_with_the_call():
    from hash_table_cache_amd import training as T

    w = T.load().hkv_train_workspace_bytes
    assert w(0, 0, 0) % 16 == 0
    assert w(1000, 0, 0) > w(10, 0, 0) and w(10, 500, 0) > w(10, 0, 0) and w(0, 0, 300) > w(0, 0, 1)


# values that stand for device addresses; every refusal below comes before any look at them
P = ctypes.c_void_p(4096)


def last():
    from hash_table_cache_amd import training as T

    return T.load().hkv_train_last_error().decode()


def logits_args(rows=4, vocab=8, dtype=0, stride=8, temperature=1.0):
    return [rows, vocab, dtype, P, stride, P, temperature]


BAD_LOGITS = [
    (dict(dtype=3), "dtype"),
    (dict(rows=1 << 31), "rows"),
    (dict(vocab=0), "vocab"),
    (dict(vocab=1 << 29, stride=1 << 29), "vocab"),
    (dict(stride=7), "logits_stride"),
    (dict(temperature=0.0), "temperature"),
    (dict(temperature=-1.0), "temperature"),
    (dict(temperature=float("nan")), "temperature"),
    (dict(temperature=float("inf")), "temperature"),
    (dict(temperature=1e-39), "temperature"),
]


@pytest.mark.parametrize("kw,needle", BAD_LOGITS)
def test_every_logits_call_refuses(kw, needle):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    L = T.load()
    a = logits_args(**kw)
    assert L.hkv_token_logprobs(*a, P, P, P, 1 << 20, None) == _native.HKV_EINVAL and needle in last()
    assert L.hkv_token_logprobs_backward(*a, P, P, P, 1 << 30, None) == _native.HKV_EINVAL and needle in last()
    assert L.hkv_preference_loss(*a, 1, P, P, .1, 0., 1., P, P, P, P, P, 1 << 30, P, 1 << 20, None) == _native.HKV_EINVAL
    assert needle in last()
    assert L.hkv_policy_loss(*a, P, P, P, P, .2, .2, 0., 1., P, P, P, P, P, 1 << 30, P, 1 << 20,
                             None) == _native.HKV_EINVAL
    assert needle in last()


@pytest.mark.parametrize("beta,smoothing,scale,pairs,needle", [
    (float("nan"), 0.0, 1.0, 1, "beta"), (0.1, -0.1, 1.0, 1, "label_smoothing"), (0.1, 1.5, 1.0, 1, "label_smoothing"),
    (0.1, float("nan"), 1.0, 1, "label_smoothing"), (0.1, 0.0, float("inf"), 1, "grad_scale"),
    (0.1, 0.0, 1.0, 1 << 30, "pairs"),
])
def test_preference_refuses(beta, smoothing, scale, pairs, needle):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    st = T.load().hkv_preference_loss(*logits_args(), pairs, P, P, beta, smoothing, scale, P, P, P, P, P, 8, P, 1 << 20,
                                      None)
    assert st == _native.HKV_EINVAL and needle in last()


@pytest.mark.parametrize("low,high,kl,scale,ref,needle", [
    (-0.1, 0.2, 0.0, 1.0, P, "clip_low"), (1.1, 0.2, 0.0, 1.0, P, "clip_low"), (0.2, -0.1, 0.0, 1.0, P, "clip_high"),
    (0.2, float("inf"), 0.0, 1.0, P, "clip_high"), (0.2, 0.2, float("nan"), 1.0, P, "kl_coef"),
    (0.2, 0.2, 0.1, 1.0, None, "ref_logp"), (0.2, 0.2, 0.0, float("nan"), P, "grad_scale"),
])
def test_policy_refuses(low, high, kl, scale, ref, needle):
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    st = T.load().hkv_policy_loss(*logits_args(), P, P, P, ref, low, high, kl, scale, P, P, P, P, P, 8, P, 1 << 20, None)
    assert st == _native.HKV_EINVAL and needle in last()


def test_clip_refuses():
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    L = T.load()
    ptrs, numel = (ctypes.c_void_p * 1)(4096), (ctypes.c_uint64 * 1)(8)
    ws = 1 << 20

    def clip(n=1, g=ptrs, c=numel, k=b"\0", max_norm=1.0):
        return L.hkv_clip_grad_norm(n, g, None, c, k, max_norm, P, P, ws, None)

    assert clip(max_norm=-1.0) == _native.HKV_EINVAL and "max_norm" in last()
    assert clip(max_norm=float("nan")) == _native.HKV_EINVAL and "max_norm" in last()
    assert clip(k=b"\7") == _native.HKV_EINVAL and "dtype" in last()
    assert clip(n=1 << 20) == _native.HKV_EINVAL and "tensors" in last()
    assert clip(g=None) == _native.HKV_EINVAL and "NULL" in last()
    assert clip(c=(ctypes.c_uint64 * 1)(1 << 50)) == _native.HKV_EINVAL and "numel" in last()


def test_host_memory_is_refused():
    from hash_table_cache_amd import _native
    from hash_table_cache_amd import training as T

    host = torch.zeros(64)
    y = torch.zeros(4, dtype=torch.int64)
    st = T.load().hkv_token_logprobs(4, 8, 0, host.data_ptr(), 8, y.data_ptr(), 1.0, host.data_ptr(), None,
                                     host.data_ptr(), 1 << 20, None)
    assert st == _native.HKV_EINVAL and "logits" in last()
    assert T.load().hkv_token_logprobs(4, 8, 0, None, 8, None, 1.0, None, None, None, 1 << 20, None) == _native.HKV_EINVAL
    assert "NULL" in last()


def test_python_checks_come_first():
    import hash_table_cache_amd as H

    x, y, f = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        H.token_logprobs(x, y)
    with pytest.raises(TypeError, match="float64"):
        H.token_logprobs(x.double(), y)
    with pytest.raises(ValueError, match="two dimensions"):
        H.policy_loss(x[None], y, f, f, f)
    with pytest.raises(ValueError, match="at least one"):
        H.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="GPU"):
        H.clip_grad_norm([x], 1.0)
