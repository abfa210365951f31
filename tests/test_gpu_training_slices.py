"""The training operators where launches are cut into slices of rows, offsets pass
32 bits, and teams are small because rows are many."""

import pytest
import torch

import training_reference as R
from conftest import gpu_available
from test_gpu_training_ops import dev, grad_tolerance

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_gradients_past_32_bits_and_one_launch():
    """Rows on both sides of 2^32 elements and of the 2^14 rows that one launch
    of the gradients in parts takes at this length; logits past the caches."""
    import hash_table_cache_amd as H

    vocab, rows = 1 << 18, (1 << 14) + 3
    pick = [0, 1, (1 << 13) - 1, 1 << 13, (1 << 14) - 1, 1 << 14, rows - 1]
    gen = torch.Generator(device=dev()).manual_seed(3)
    kept = torch.randn(len(pick), vocab, dtype=torch.bfloat16, device=dev(), generator=gen)
    y = torch.full((rows,), -1, dtype=torch.int64, device=dev())
    y[pick] = torch.tensor([5, 77, 1000, vocab - 1, 3, vocab // 2, 9], device=dev())
    want = R.Rows(kept, y[pick], 1.0)
    x = torch.empty((rows, vocab), dtype=torch.bfloat16, device=dev())

    def fresh():  # rows without a label hold what their gradient must replace
        x.fill_(1.0)
        x[pick] = kept

    def rest_is_zero():
        x[pick] = 0.0
        return not any(bool(x[a:a + 2048].any()) for a in range(0, rows, 2048))

    fresh()
    logp, lse = H.token_logprobs(x, y)
    R.assert_near(logp[pick], want.logp, R.LOGP + want.logp.abs() * R.EPS, "logp")
    R.assert_near(lse[pick], want.lse, R.LOGP + want.lse.abs() * R.EPS, "lse")
    g = torch.linspace(1.0, 2.0, len(pick))
    g_rows = torch.ones(rows, device=dev())
    g_rows[pick] = g.to(dev())
    z = R.f64(kept) - R.f64(lse[pick])[:, None]
    at = torch.arange(len(pick)), y[pick].cpu()
    d = -torch.exp(z)
    d[at] = -torch.expm1(z[at])
    grad = H.token_logprobs_backward(x, y, lse, g_rows, grad_out=x)
    ref = g.double()[:, None] * d
    R.assert_near(grad[pick], ref, ref.abs() * (R.GRAD + R.half_step(x.dtype)) + R.TINY[x.dtype], "backward")
    assert rest_is_zero()

    cu = torch.tensor([0, 2, 1 << 13, 1 << 14, rows])
    ref_logp = torch.zeros(rows, device=dev())
    ref_logp[pick] = (want.logp - torch.linspace(-0.5, 0.9, len(pick))).float().to(dev())
    seq = torch.tensor([0, 0, 1, 2, 2, 3, 3])
    ratio = want.logp - R.f64(ref_logp[pick])
    rewards = 0.25 * torch.zeros(4, dtype=torch.float64).index_add_(0, seq, ratio)
    m = rewards[0::2] - rewards[1::2]
    c = 0.25 * (torch.sigmoid(m) - 1) / 2 * 64.0
    g = torch.where(seq % 2 == 0, c[seq // 2], -c[seq // 2])
    fresh()
    out = H.preference_loss(x, y, cu.to(dev()), ref_logp, beta=0.25, grad_scale=64.0, grad_out=x)
    d_reward = 0.25 * 2 * R.LOGP
    R.assert_near(out.rewards, rewards, d_reward + rewards.abs() * R.EPS, "rewards")
    loss = torch.nn.functional.softplus(-m).mean()
    R.assert_near(out.loss, loss, 2 * d_reward + loss * R.EPS, "loss")
    delta = torch.full((len(pick),), 64.0 * 0.25 / 2 * 2 * d_reward / 4, dtype=torch.float64) + g.abs() * 4 * R.EPS
    R.assert_near(out.grad[pick], want.grad(g), grad_tolerance(want, g, x.dtype, delta), "pair grad")
    assert rest_is_zero()


def test_more_rows_than_a_launch():
    """2^25 rows of short lists are one launch of the smallest teams; the rows
    after them go by a second one, in every operator."""
    import hash_table_cache_amd as H

    vocab, rows = 8, (1 << 25) + 5
    gen = torch.Generator(device=dev()).manual_seed(6)
    x = torch.randn(rows, vocab, device=dev(), generator=gen).to(torch.bfloat16)
    y = torch.randint(0, vocab, (rows,), device=dev(), generator=gen)
    y[::7] = -1
    y[-5:] = torch.tensor([0, 7, -1, 3, 4], device=dev())
    pick = torch.cat([torch.arange(0, 20), torch.arange((1 << 25) - 20, rows)])
    on = pick.to(dev())
    want = R.Rows(x[on], y[on], 1.0)
    near = R.LOGP + want.logp.abs() * R.EPS
    logp, lse = H.token_logprobs(x, y)
    R.assert_near(logp[on], want.logp, near, "logp")
    # all rows against torch in float32: two results of that type, a few steps of numbers up to 8 apart
    plain = torch.log_softmax(x.float(), 1).gather(1, y.clamp(min=0)[:, None])[:, 0].masked_fill_(y < 0, 0.0)
    assert float((logp - plain).abs().max()) < 64 * 8 * R.EPS
    ones = torch.ones(rows, device=dev())
    back = H.token_logprobs_backward(x, y, lse, ones)
    z = R.f64(x[on]) - R.f64(lse[on])[:, None]
    at = torch.arange(len(pick)), y[on].cpu().clamp(min=0)
    d = -torch.exp(z)
    d[at] = -torch.expm1(z[at])
    d[~want.counts] = 0.0
    R.assert_near(back[on], d, d.abs() * (R.GRAD + R.half_step(x.dtype)) + R.TINY[x.dtype], "backward")
    weights = ones / rows
    pol = H.policy_loss(x, y, logp, ones, weights, grad_scale=float(rows))
    live = int((y >= 0).sum())
    # the ratio is 1 but for the rounding of the old log-probability, at most 4 eps and of either sign
    assert float(pol.loss) == pytest.approx(-live * float(weights[0]), abs=8 * R.EPS)
    g = torch.where(want.counts, -torch.exp(want.logp - R.f64(logp[on])), 0.0)
    delta = g.abs() * (R.LOGP + 8 * R.EPS)
    R.assert_near(pol.grad[on], want.grad(g), grad_tolerance(want, g, x.dtype, delta), "policy grad")
    assert int((pol.grad != 0).any(1).sum()) == live  # every row was written, and only those with a label
    cu = torch.tensor([0, 1 << 24, 1 << 25, (1 << 25) + 2, rows], device=dev())
    ref = logp - 2.0 ** -24
    pref = H.preference_loss(x, y, cu, ref, beta=0.5, grad_scale=float(rows))
    seq = torch.stack([(logp - ref)[a:b].masked_fill(y[a:b] < 0, 0.0).double().sum()
                       for a, b in ((0, 1 << 24), (1 << 24, 1 << 25), (1 << 25, (1 << 25) + 2), ((1 << 25) + 2, rows))]).cpu()
    # what the old logp lost to rounding is summed as well: half a step of up to 8, each
    n = torch.tensor([1 << 24, 1 << 24, 2, 3], dtype=torch.float64)
    R.assert_near(pref.rewards, 0.5 * seq, 0.5 * n * (R.LOGP + 8 * R.EPS), "rewards")
    m = R.f64(pref.rewards)[0::2] - R.f64(pref.rewards)[1::2]
    c = 0.5 * (torch.sigmoid(m) - 1) / 2 * rows
    s = torch.bucketize(pick, cu.cpu(), right=True) - 1
    g = torch.where(s % 2 == 0, c[s // 2], -c[s // 2])
    g = torch.where(want.counts, g, 0.0)
    delta = g.abs() * 8 * R.EPS + 0.5 / 2 * rows * R.f64(pref.rewards).abs().sum() * R.EPS / 4
    R.assert_near(pref.grad[on], want.grad(g), grad_tolerance(want, g, x.dtype, delta), "pair grad")
    assert int((pref.grad != 0).any(1).sum()) == live


@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 8), (torch.float16, 1003), (torch.bfloat16, 4099),
                                         (torch.float32, 7001), (torch.bfloat16, 30011)])
def test_gradients_of_thousands_of_rows(dtype, vocab):
    """Backward and preference gradients among thousands of rows, from the
    formula alone: rewards, coefficients and elements."""
    import hash_table_cache_amd as H

    rows, tau = 4099, 1.25
    gen = torch.Generator(device=dev()).manual_seed(vocab)
    x = torch.randn(rows, vocab, device=dev(), generator=gen).mul_(3.0).to(dtype)
    y = torch.randint(0, vocab, (rows,), device=dev(), generator=gen)
    y[::9] = -1
    logp = torch.empty(rows, dtype=torch.float64)
    for a in range(0, rows, 512):
        z = torch.log_softmax(x[a:a + 512].double() / tau, 1)
        logp[a:a + 512] = z.gather(1, y[a:a + 512].clamp(min=0)[:, None])[:, 0].masked_fill(y[a:a + 512] < 0, 0.0).cpu()
    pick = torch.cat([torch.arange(0, 20), torch.arange(1990, 2010), torch.arange(rows - 8, rows)])
    on = pick.to(dev())
    want = R.Rows(x[on], y[on], tau)
    cu = torch.tensor([0, 2000, rows])
    moved = torch.where(torch.arange(rows) < 2000, -0.005, 0.005).double()
    ref = (logp + moved + 0.05 * torch.randn(rows, generator=torch.Generator().manual_seed(1)).double()).float()
    ratio = torch.where(y.cpu() >= 0, logp - ref.double(), 0.0)
    rewards = 0.1 * torch.stack([ratio[:2000].sum(), ratio[2000:].sum()])
    out = H.preference_loss(x, y, cu.to(dev()), ref.to(dev()), temperature=tau, grad_scale=8.0)
    d_reward = 0.1 * torch.tensor([2000.0, rows - 2000.0], dtype=torch.float64) * R.LOGP
    R.assert_near(out.rewards, rewards, d_reward + rewards.abs() * R.EPS, "rewards")
    c = 0.1 * (torch.sigmoid(rewards[0] - rewards[1]) - 1) * 8.0
    g = torch.where(pick < 2000, c, -c)
    delta = 0.1 * 8.0 * d_reward.sum() / 4 + g.abs() * 4 * R.EPS
    R.assert_near(out.grad[on], want.grad(g), grad_tolerance(want, g, dtype, delta), "pair grad")
    assert not bool(out.grad[y < 0].any())

    lse = H.token_logprobs(x, y, temperature=tau)[1]
    g = torch.linspace(-2.0, 2.0, rows)
    back = H.token_logprobs_backward(x, y, lse, g.to(dev()), temperature=tau)
    z = R.f64(x[on]) / want.tau - R.f64(lse[on])[:, None]
    at = torch.arange(len(pick)), y[on].cpu().clamp(min=0)
    want.d = -torch.exp(z)
    want.d[at] = -torch.expm1(z[at])
    want.d[~want.counts] = 0.0
    ref = want.grad(g[pick].double())
    R.assert_near(back[on], ref, ref.abs() * (R.GRAD + R.half_step(dtype)) + R.TINY[dtype], "backward")
    assert not bool(back[y < 0].any())
