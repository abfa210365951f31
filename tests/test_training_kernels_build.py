"""What the training library's kernels are compiled to: gfx950, no packed fp32
arithmetic, and nothing kept in memory for want of registers."""

import subprocess

import pytest

from hash_table_cache_amd import build as hb

SOURCES = [s for s in hb.TRAIN_SOURCES if str(s).endswith(".hip")]


@pytest.mark.parametrize("source", SOURCES, ids=lambda s: s.name)
def test_no_packed_fp32_and_no_spills(source):
    out = subprocess.run([hb.hipcc(), *hb.compile_flags(), "--offload-device-only", "-S", "-x", "hip", str(source), "-o", "-"],
                         capture_output=True, text=True, check=True)
    assert "gfx950" in out.stdout
    for op in ("add", "mul", "fma"):
        assert "v_pk_" + op + "_f32" not in out.stdout
    assert "scratch_store" not in out.stdout


def test_every_source_is_built():
    assert {s.name for s in SOURCES} == {p.name for p in hb.CSRC.glob("hkv_train_*.hip")}
