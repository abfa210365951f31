"""The policy loss as a weighted sum, against its formula."""

import math

import pytest
import torch

import training_reference as R
from conftest import gpu_available
from test_gpu_training_ops import dev, grad_tolerance, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("rows,vocab", [(1, 8), (41, 8), (41, 1000), (300, 2049), (259, 70001), (3, 140001), (20001, 40)])
@pytest.mark.parametrize("kl_coef", [0.0, 0.2])
def test_weighted_policy_loss(rows, vocab, kl_coef):
    """The sum of the policy loss with weights that all differ, in every kind
    of launch; what mistakes in it would give lies outside the tolerance."""
    import hash_table_cache_amd as H

    x, y = make(rows, vocab, torch.float32, 500 + vocab, special=False)
    if rows > 16:  # rows left out, and one that is half masked
        y[5], x[7] = -1, -torch.inf
        x[9, :vocab // 2], y[9] = -torch.inf, vocab - 1
    want = R.Rows(x, y, 1.0)
    gen = torch.Generator().manual_seed(3)
    d = 0.3 * torch.randn(rows, generator=gen).double()
    for border in (math.log(1 - 0.2), math.log(1 + 0.3)):  # none on a bound
        d = torch.where((d - border).abs() < 1e-3, d + 2e-3, d)
    old = (want.logp - d).float()
    ref = (want.logp + 0.5 * torch.randn(rows, generator=gen).double()).float()
    adv = torch.randn(rows, generator=gen) + 0.3
    w = (0.5 + torch.rand(rows, generator=gen)) / rows
    args = (0.2, 0.3, kl_coef, 32.0)
    total, loss, kl, g = R.policy(want, old, adv, w, ref, *args)
    r, e = torch.exp(want.logp - old.double()), torch.exp(ref.double() - want.logp)
    slope = torch.where(want.counts, (r * adv.double()).abs() + kl_coef * (e + 1), 0.0)
    tol = float((slope * R.LOGP * w.double()).sum() + total.abs() * R.EPS)
    assert math.isfinite(float(total)) and float(total) != 0.0
    wrong = [R.policy(want, old, adv, w + 0.01 / rows, ref, *args)[0], R.policy(want, old, adv, w, ref, 0.2, 0.3, 0.01, 1.0)[0]]
    if rows > 1:
        wrong += [R.policy(want, old, adv, w.roll(1), ref, *args)[0], (w[:-1].double() * loss[:-1]).sum()]
    assert all(abs(float(v - total)) > 2 * tol for v in wrong)
    dargs = [t.to(dev()) for t in (old, adv, w, ref)]
    got = H.policy_loss(x, y, *dargs, clip_high=0.3, kl_coef=kl_coef, grad_scale=32.0)
    value = H.policy_loss(x, y, *dargs, clip_high=0.3, kl_coef=kl_coef, with_grad=False)
    for out in (got, value):
        R.assert_near(out.loss, total, tol, "loss")
        R.assert_near(out.token_loss, loss, slope * R.LOGP + loss.abs() * R.EPS, "token_loss")
    some = slice(None) if rows <= 300 else slice(0, 300)
    delta = slope * R.LOGP * w.double() * 32.0 + g.abs() * 4 * R.EPS
    R.assert_near(got.grad[some], want.grad(g)[some], grad_tolerance(want, g, torch.float32, delta)[some], "grad")
    assert int((got.grad != 0).any(1).sum()) == int((g != 0).sum())


def test_masked_label_with_a_reference():
    """A label whose own logit is -inf: its divergence is NaN and stays in kl_out unless the loss counts it."""
    import hash_table_cache_amd as H

    rows, vocab = 20, 50
    x, y = make(rows, vocab, torch.float32, 31, special=False)
    x[3, y[3]] = -torch.inf
    want = R.Rows(x, y, 1.0)
    old = want.logp.nan_to_num(0.0, 0.0, -3.0).float().to(dev())
    ones = torch.ones(rows, device=dev())
    got = H.policy_loss(x, y, old, ones, ones, old)
    assert math.isnan(float(got.kl[3])) and int(got.kl.isnan().sum()) == 1
    assert float(got.logp[3]) == -math.inf and float(got.token_loss[3]) == 0.0 and not bool(got.grad[3].any())
    # every other ratio is 1 but for the rounding of the old log-probability, of at most 8 units
    assert float(got.loss) == pytest.approx(-(rows - 1), rel=8 * R.EPS)
    assert math.isnan(float(H.policy_loss(x, y, old, ones, ones, old, kl_coef=0.1).loss))
    y[3] = -1
    got = H.policy_loss(x, y, old, ones, ones, old, kl_coef=0.1)
    assert float(got.loss) == pytest.approx(-(rows - 1), rel=8 * R.EPS) and not bool(got.kl.isnan().any())
