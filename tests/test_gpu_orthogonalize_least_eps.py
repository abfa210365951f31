"""The smallest eps that 64 bits hold: zeros still give zeros, and a matrix of the
smallest numbers its directions."""

import pytest
import torch

import polar_reference as P
import training_reference as R
from conftest import gpu_available
from test_gpu_orthogonalize import dev, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("eps", [5e-324, 1e-310, 1e-300])
@pytest.mark.parametrize("shape", [(20, 30), (50, 700), (100, 130)])
def test_zeros(shape, eps):
    import hash_table_cache_amd as H

    for dtype in (torch.float32, torch.bfloat16):
        got, low = H.orthogonalize([torch.zeros(shape, dtype=dtype, device=dev()),
                                    (make(*shape, torch.float32, 1) * 2.0 ** -100).to(dtype)], eps=eps)
        assert not bool(got.any())
        P.assert_polar(low, R.f64((make(*shape, torch.float32, 1) * 2.0 ** -100).to(dtype)), eps=eps)
        w, m = make(*shape, dtype, 2), torch.zeros(shape, device=dev())
        before = w.clone()
        H.muon_update([w], [torch.zeros_like(w)], [m], 0.1, eps=eps)
        assert torch.equal(w, before)
