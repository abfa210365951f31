"""Which matrices may lie in one buffer: those that share no element, whatever
their numbers of rows, are separate ones; those that do are refused."""

import pytest
import torch

import polar_reference as P
import training_reference as R
from conftest import gpu_available
from test_gpu_orthogonalize import dev, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

# views of a buffer of 50 rows of 180
APART = {
    "a row beside a column block": lambda w: (w[:, :60], w[7:8, 100:180]),
    "a row before a column block": lambda w: (w[0:1, :100], w[:, 100:180]),
    "the last row's end": lambda w: (w[:, :60], w[49:50, 60:]),
    "rows of their own": lambda w: (w[3:4], w[4:5], w[5:20], w[20:21, :90], w[20:21, 90:]),
    "every second row beside all rows": lambda w: (w[0::2, :50], w[:, 50:]),
    "every second row and every third": lambda w: (w[0::2, :50], w[0::3, 50:90], w[1::2, :50]),
    "a column beside others": lambda w: (w[:, 7:8], w[:, :7], w[:, 8:], ),
}
SHARED = {
    "a row across a column block": lambda w: (w[:, :60], w[7:8, 59:100]),
    "a row into the next one's block": lambda w: (w[:, :60], w.view(-1)[7 * 180 + 100:8 * 180 + 1].view(1, -1)),
    "one element": lambda w: (w[:, :60], w[49:50, 59:60]),
    "the same row": lambda w: (w[3:4], w[3:4]),
    "every second row and every third": lambda w: (w[0::2, :50], w[0::3, 40:90]),
}


@pytest.mark.parametrize("which", APART)
def test_apart(which):
    import hash_table_cache_amd as H

    w = make(50, 180, torch.float32, 1).contiguous()
    before = w.clone()
    parts, old = APART[which](w), APART[which](before)
    H.orthogonalize(parts, out=parts)
    taken = torch.zeros_like(w)
    for i, (p, o, t) in enumerate(zip(parts, old, APART[which](taken))):
        P.assert_polar(p, R.f64(o), what=f"{which} {i}")
        t.fill_(1.0)
    assert torch.equal(w[taken == 0], before[taken == 0])


@pytest.mark.parametrize("which", SHARED)
def test_shared(which):
    import hash_table_cache_amd as H

    w = make(50, 180, torch.float32, 1).contiguous()
    before = w.clone()
    parts = SHARED[which](w)
    with pytest.raises(H.HkvError, match="overlap"):
        H.orthogonalize(parts, out=parts)
    momenta = [torch.zeros(p.shape, device=dev()) for p in parts]
    with pytest.raises(H.HkvError, match="overlap"):
        H.muon_update(parts, [m.clone() for m in momenta], momenta, 0.1)
    assert torch.equal(w, before)
