"""Matrices written in place count as modified: a backward pass that saved one
fails instead of taking its new values, and one that did not goes on."""

import pytest
import torch

from conftest import gpu_available
from test_gpu_orthogonalize import dev, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def versions(ts):
    return [t._version for t in ts]


def test_backward_through_updated_weights():
    import hash_table_cache_amd as H

    w = [torch.nn.Parameter(make(40, 60, torch.float32, i)) for i in range(2)]
    m = [torch.zeros(40, 60, device=dev()) for _ in w]
    x = torch.randn(40, device=dev(), requires_grad=True)
    first, second = (x @ w[0]).sum(), (x @ w[1]).sum()  # each saved its weight, for the gradient of x
    g = [make(40, 60, torch.float32, 5 + i) for i in range(2)]
    H.muon_update(w[:1], g[:1], m[:1], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        first.backward()
    second.backward()  # nothing of its was written
    assert torch.allclose(x.grad, w[1].detach().sum(1), atol=1e-6)
    # after the step a new pass sees the new weights
    x.grad = None
    (x @ w[0]).sum().backward()
    assert torch.allclose(x.grad, w[0].detach().sum(1), atol=1e-6)


def test_which_tensors_count():
    import hash_table_cache_amd as H

    w, g, m = ([make(30, 50, torch.bfloat16, i) for i in range(2)], [make(30, 50, torch.bfloat16, 3 + i) for i in range(2)],
               [torch.zeros(30, 50, device=dev()) for _ in range(2)])
    before = versions(w + m), versions(g)
    H.muon_update(w, g, m, 0.1)
    assert [b - a for a, b in zip(before[0], versions(w + m))] == [1] * 4 and versions(g) == before[1]
    out = [torch.empty_like(x) for x in g]
    H.orthogonalize(g, out=out)
    assert all(v >= 1 for v in versions(out)) and versions(g) == before[1]
    H.orthogonalize(g, out=g)
    assert versions(g) == [v + 1 for v in before[1]]
    with pytest.raises(H.HkvError):  # a refused call writes nothing
        H.muon_update(w, g, m, 0.1, momentum=1.5)
    assert [b - a for a, b in zip(before[0], versions(w + m))] == [1] * 4


def test_in_inference_mode():
    import hash_table_cache_amd as H

    with torch.inference_mode():
        w, g, m = make(30, 50, torch.float32, 1), make(30, 50, torch.float32, 2), torch.zeros(30, 50, device=dev())
        before = w.clone()
        H.muon_update([w], [g], [m], 0.1)
        assert not torch.equal(w, before)
