"""The training operators in 64 bits on the CPU, from their formulas, and the
error bounds that the 32-bit kernels are held to.

Bounds. eps = 2^-24 is half a step of float32. The sum S of a row's
exponentials: a term with exponent -a carries at most 2 a eps from its
argument (weight e^-a, so under 2 eps of the sum), 2 eps from the exponential,
up to 5 eps from the sum of up to 32 terms, and 4 eps for each of the few times
that a thread finds a larger maximum: LOGP = 32 eps covers S, and with it logp, absolutely.
An element of the gradient adds 3 a eps (a <= 60: what is smaller than e^-60 is
covered by the absolute part) and a few roundings: GRAD = 220 eps, relatively.
Then the rounding to the output's type, half its step.
"""

import torch

EPS = torch.finfo(torch.float32).eps / 2
LOGP = 32 * EPS
GRAD = 220 * EPS
# half the smallest step of each type (results below its normal range)
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def f64(t):
    return t.detach().cpu().double()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Rows:
    """Row-wise softmax of logits: counts (rows not left out), lse, logp, d
    (1[label] - p), all in 64 bits."""

    def __init__(self, x, labels, temperature):
        tau = float(torch.tensor(temperature, dtype=torch.float32))
        self.tau = tau
        z = f64(x) / tau
        y = labels.detach().cpu()
        rows, vocab = z.shape
        empty = (z == -torch.inf).all(1)
        bad = (y >= vocab) | (z.isnan() | (z == torch.inf)).any(1)
        self.counts = (y >= 0) & ~(empty & ~bad)
        bad &= y >= 0
        at = torch.where(y >= vocab, torch.zeros_like(y), y.clamp(min=0))
        ok = self.counts & ~bad
        safe = torch.where(ok[:, None], z, torch.zeros_like(z))
        # from each row's maximum: beside 1e38 even 64 bits hold no log(vocab)
        top = safe.amax(1)
        safe = safe - top[:, None]
        self.lse = torch.logsumexp(safe, 1)
        label = safe.gather(1, at[:, None])[:, 0]
        # the other terms' sum apart, so that nearly certain rows lose nothing
        others = safe.clone()
        others[torch.arange(rows), at] = -torch.inf
        rest = torch.logsumexp(others, 1) if vocab > 1 else torch.full((rows,), -torch.inf, dtype=torch.float64)
        self.logp = torch.where(label >= rest, -torch.log1p(torch.exp(rest - label)), label - self.lse)
        p = torch.exp(safe - self.lse[:, None])
        self.d = -p
        self.d[torch.arange(rows), at] = torch.exp(rest - self.lse)
        self.lse = self.lse + top
        nan = torch.tensor(torch.nan, dtype=torch.float64)
        self.lse = torch.where(bad, nan, torch.where(y < 0, 0.0, torch.where(self.counts, self.lse, -torch.inf)))
        self.logp = torch.where(bad, nan, torch.where(self.counts, self.logp, 0.0))
        self.d = torch.where(bad[:, None], nan, torch.where(self.counts[:, None], self.d, 0.0))

    def grad(self, g):
        """g / tau (1[label] - p); rows with g = 0 are zeros."""
        out = (g / self.tau)[:, None] * self.d
        return torch.where((g == 0)[:, None], 0.0, out)


def preference(rows, cu, ref, beta, smoothing, scale):
    beta, smoothing, scale = (float(torch.tensor(v, dtype=torch.float32)) for v in (beta, smoothing, scale))
    ratio = rows.logp - (0.0 if ref is None else f64(ref))
    ratio = torch.where(rows.counts, ratio, 0.0)
    n = ratio.numel()
    cu = cu.cpu().tolist()
    pairs = len(cu) // 2
    rewards = torch.stack([beta * ratio[cu[s]:cu[s + 1]].sum() for s in range(2 * pairs)]) if pairs else torch.zeros(0).double()
    m = rewards[0::2] - rewards[1::2]
    losses = torch.zeros_like(m)
    if smoothing != 1.0:
        losses = losses + (1 - smoothing) * torch.nn.functional.softplus(-m, threshold=1e9)
    if smoothing != 0.0:
        losses = losses + smoothing * torch.nn.functional.softplus(m, threshold=1e9)
    c = beta * (torch.sigmoid(m) - 1 + smoothing) / max(pairs, 1) * scale
    g = torch.zeros(n, dtype=torch.float64)
    for s in range(2 * pairs):
        g[cu[s]:cu[s + 1]] = c[s // 2] if s % 2 == 0 else -c[s // 2]
    loss = losses.mean() if pairs else torch.zeros(()).double()
    return loss, losses, rewards, g


def policy(rows, old, adv, weights, ref, low, high, kl_coef, scale):
    low, high, kl_coef, scale = (float(torch.tensor(v, dtype=torch.float32)) for v in (low, high, kl_coef, scale))
    old, adv, weights = f64(old), f64(adv), f64(weights)
    r = torch.exp(rows.logp - old)
    free, bound = r * adv, r.clamp(1 - low, 1 + high) * adv
    loss = -torch.minimum(free, bound)
    g = torch.where(free <= bound, -free, torch.where(free.isnan(), free, 0.0))
    kl = torch.zeros_like(loss)
    if ref is not None:
        d = f64(ref) - rows.logp
        kl = torch.expm1(d) - d
        if kl_coef:
            loss = loss + kl_coef * kl
            g = g - kl_coef * torch.expm1(d)
    loss, kl, g = (torch.where(rows.counts, v, 0.0) for v in (loss, kl, g))
    total = torch.where(loss != 0, weights * loss, 0.0).sum()
    return total, loss, kl, g * weights * scale


def assert_near(got, want, tol, what):
    """|got - want| <= tol elementwise; NaN where NaN, equal infinities; what
    is past the range of got's type has to be an infinity there."""
    want = torch.where(want.abs() > torch.finfo(got.dtype).max, want.sign() * torch.inf, want)
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    fine = want.isfinite()
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), f"{what}: infinities differ"
    off = (got - want).abs()[fine]
    tol = torch.as_tensor(tol, dtype=torch.float64).expand(want.shape)[fine]
    if off.numel():
        worst = int((off - tol).argmax())
        assert bool((off <= tol).all()), f"{what}: off by {off[worst]:.3e}, {tol[worst]:.3e} allowed, at {fine.nonzero()[worst].tolist()}"
