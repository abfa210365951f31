"""How exactly a row's sum is held: log-probabilities before their rounding to
float32, which differences of them (the divergence, rewards) show."""

import pytest
import torch

import training_reference as R
from conftest import gpu_available
from test_gpu_training_ops import dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def step(v):
    """The distance of float32 numbers at |v|."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -126))) - 23)


@pytest.mark.parametrize("vocab,tau", [(60, 1.0), (1000, 1.0), (1445, 0.5), (20000, 0.75)])
def test_sums_add_nothing_to_the_exponentials_error(vocab, tau):
    """Rewards of single rows are logp - ref_logp in 64 bits until their own
    rounding. What they are off by is each exponential's part of the sum times
    the roundings of its argument and of itself: independent, each uniform over
    a step, a quarter more for an exponential that may be a whole step off.
    Partial sums in 32 bits would add as much again."""
    import hash_table_cache_amd as H

    rows = 8192
    gen = torch.Generator(device=dev()).manual_seed(vocab)
    x = torch.randn(rows, vocab, device=dev(), generator=gen) * 2.5
    y = torch.randint(0, vocab, (rows,), device=dev(), generator=gen)
    logp = torch.empty(rows, dtype=torch.float64, device=dev())
    variance = torch.empty_like(logp)
    for a in range(0, rows, 1024):
        z, at = x[a:a + 1024].double(), y[a:a + 1024, None]
        logp[a:a + 1024] = torch.log_softmax(z / tau, 1).gather(1, at)[:, 0]
        rest = 1.0 - logp[a:a + 1024].exp()
        z.scatter_(1, at, -1e3)  # the label is no part of the sum
        z -= z.amax(1, keepdim=True)
        share = torch.softmax(z / tau, 1)
        argument = (step(z) / tau) ** 2 + (step(z / tau / 0.6931471805599453) * 0.6931471805599453) ** 2
        variance[a:a + 1024] = (share ** 2 * (argument + (2 * R.EPS) ** 2)).sum(1) / 12 * rest ** 2
    allowed = 1.25 * float(variance.mean().sqrt())
    ref = logp.float()
    cu = torch.arange(rows + 1, device=dev())
    got = H.preference_loss(x, y, cu, ref, beta=1.0, temperature=tau, with_grad=False).rewards
    off = got.double() - (logp - ref.double())
    rms = float(off.square().mean().sqrt())
    assert rms < allowed, f"{rms / R.EPS:.3f} against {allowed / R.EPS:.3f}, in 2^-24"
