"""Where the training operators take and leave their data: gradients beside
their logits, results that belong to no other tensor."""

import pytest
import torch

import training_reference as R
from conftest import gpu_available
from test_gpu_training_ops import TYPES, dev, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,gap", [(1, 0), (7, 0), (300, 1), (1025, 0), (5003, 3), (20001, 0)])
def test_gradient_in_other_columns(vocab, gap, dtype):
    """Logits and gradient are different columns of the same rows: no element is shared."""
    import hash_table_cache_amd as H

    rows = 9
    gen = torch.Generator().manual_seed(vocab)
    y = torch.randint(0, vocab, (rows,), generator=gen).to(dev())
    y[4] = -1
    ones = torch.ones(rows, device=dev())
    cu = torch.tensor([0, 4, 9], device=dev())
    for x_first in (True, False):
        left, right = slice(1, 1 + vocab), slice(1 + vocab + gap, 1 + 2 * vocab + gap)
        wide = torch.randn(rows, 2 * vocab + gap + 2, generator=gen).to(dtype).to(dev())
        x, out = (wide[:, left], wide[:, right]) if x_first else (wide[:, right], wide[:, left])
        want = R.Rows(x, y, 1.0)
        f = (want.logp + 0.05).float().to(dev())
        lse = want.lse.float().to(dev())
        for call in (lambda o: H.token_logprobs_backward(x, y, lse, ones, grad_out=o),
                     lambda o: H.preference_loss(x, y, cu, f, grad_out=o).grad,
                     lambda o: H.policy_loss(x, y, f, ones, ones, grad_out=o).grad):
            apart, before = call(None), wide.clone()
            call(out)
            near = 2 * (R.GRAD + R.half_step(dtype)) * R.f64(apart).abs() + R.TINY[dtype]  # rows may be cut elsewhere
            R.assert_near(out, R.f64(apart), near, "grad")
            out.copy_(before[:, right] if x_first else before[:, left])
            assert torch.equal(wide, before)  # nothing else was written


def test_columns_that_share_elements_are_refused():
    import hash_table_cache_amd as H

    rows, vocab = 5, 40
    y = torch.zeros(rows, dtype=torch.int64, device=dev())
    f = torch.zeros(rows, device=dev())
    wide = torch.zeros(rows, 2 * vocab + 3, device=dev())
    x = wide[:, :vocab]
    flat = torch.zeros(rows * 2 * vocab + vocab, device=dev())
    lines = flat[:rows * 2 * vocab].view(rows, 2 * vocab)[:, :vocab]
    for logits, out in ((x, wide[:, 1:vocab + 1]), (x, wide[:, vocab - 1:2 * vocab - 1]),
                        (wide[:, 1:vocab + 1], x), (wide[:, 2 * vocab + 3 - vocab:], wide[:, vocab:2 * vocab]),
                        # rows of another stride, and one row further with the end in the next row's logits
                        (lines, flat[vocab:vocab + rows * vocab].view(rows, vocab)),
                        (lines, flat[vocab + 1:vocab + 1 + rows * 2 * vocab - vocab].as_strided((rows, vocab), (2 * vocab, 1)))):
        with pytest.raises(H.HkvError, match="overlaps"):
            H.policy_loss(logits, y, f, f, f, grad_out=out)
    assert not bool(wide.any()) and not bool(flat.any())


@pytest.mark.parametrize("rows", [1, 40, 100])
def test_results_stand_alone(rows):
    """Every result has memory of its own, of its own size (a kept logp keeps
    nothing else), and writing into one leaves what autograd saved of another."""
    import hash_table_cache_amd as H

    x, y = make(rows, 60, torch.float32, 11, special=False)
    f = torch.zeros(rows, device=dev())
    cu = torch.tensor([0, rows // 2, rows], device=dev())
    pref = H.preference_loss(x, y, cu, f)
    pol = H.policy_loss(x, y, f, f + 1, f + 1, f, kl_coef=0.1)
    logp, lse = H.token_logprobs(x, y)
    for results in ((logp, lse), pref, pol):
        assert len({t.untyped_storage().data_ptr() for t in results}) == len(results)
        for t in results:
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size() and t.storage_offset() == 0
    for saved, other in ((logp, lse), (pref.logp, pref.rewards), (pol.logp, pol.token_loss)):
        p = torch.ones(rows, device=dev(), requires_grad=True)
        loss = (p * saved).sum()
        other.mul_(2.0)
        loss.backward()
        assert torch.equal(p.grad, saved)


@pytest.mark.parametrize("dtype,rows,vocab", [(torch.float32, 63, 1 << 16), (torch.float32, 64, 65541), (torch.float32, 63, 65540),
                                              (torch.bfloat16, 1, 1 << 17), (torch.float16, 3, 131081)])
def test_workspace_of_logprobs(dtype, rows, vocab):
    """The rule by which log-probabilities go without a workspace is the library's own, on both sides of its borders."""
    import hash_table_cache_amd as H

    x, y = make(rows, vocab, dtype, 12, special=False)
    logp, lse = H.token_logprobs(x, y)
    want = R.Rows(x, y, 1.0)
    R.assert_near(logp, want.logp, R.LOGP + want.logp.abs() * R.EPS, "logp")
    L = H.training.load()
    stream = torch.cuda.current_stream().cuda_stream
    args = (rows, vocab, H.training.KINDS[dtype], x.data_ptr(), vocab, y.data_ptr(), 1.0, logp.data_ptr(), None, None, 0, stream)
    few_long = rows < 64 and vocab * x.element_size() // 16 > 1 << 14
    logp.fill_(7.0)
    assert (L.hkv_token_logprobs(*args) == 0) == (not few_long)
    if few_long:
        assert "workspace" in L.hkv_train_last_error().decode() and bool((logp == 7.0).all())
    else:
        R.assert_near(logp, want.logp, R.LOGP + want.logp.abs() * R.EPS, "logp")
