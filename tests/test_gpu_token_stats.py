"""Token statistics against their formulas in 64 bits: log-probability, entropy
and largest logits of rows, and the gradient through the first two.

Bound of the entropy H = log T + sum p a, a the distance from the row's maximum
in nats (eps = 2^-24). An exponent is off by 3 a eps, so a term a p by
(3 a + 6) a p eps; sums of up to 32 terms, rescaling to a larger maximum and
the error of T (32 eps, as for log-probabilities) add less than 64 eps of
sum p a and 32 eps. Then half a step of float32.

Bound of the gradient p (g + h (z + H)) / tau: p is off by GRAD relatively, which
covers the 3 |z| eps of exponents down to -60, and by 3 |z| eps past it; below
float32's normal range p is 0, off by up to 2^-126, which g + h (z + H) multiplies.
z is off by 3 eps |z|, its sum with H and the product by a few eps of their sizes.
1 / tau is a float and a second one for what is missing, at most a step of the
first, 2^-23 / tau, and itself off by 2^-24 of its size: 2^-47 |x / tau| more of z,
which shows where z is nearly 0. Then half a step of the type.
"""

import math

import pytest
import torch

import training_reference as R
from conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

TYPES = [torch.float32, torch.bfloat16, torch.float16]
VOCABS = [1, 2, 7, 8, 9, 64, 100, 511, 513, 1000, 2049, 8195, 40009]


def dev():
    return torch.device("cuda", 0)


def make(rows, vocab, dtype, seed, pad=0):
    """Logits with the rows that go wrong among ordinary ones, and labels."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab + pad, generator=gen) * 3.0).to(dtype)
    y = torch.randint(0, vocab, (rows,), generator=gen)
    x[torch.arange(rows), y] += 3.0
    if rows >= 20:
        x[1] = -torch.inf  # nothing left
        x[2, :vocab] = -torch.inf  # one candidate left, the label
        x[2, y[2]] = 1.5
        x[3, y[3]] = -torch.inf  # the label masked beside others
        y[4] = -100  # left out, with NaN among its logits
        x[4, 0] = torch.nan
        x[5, y[5]] = 40.0  # nearly certain
        x[6, : vocab // 2] = -torch.inf  # half masked
        x[7] = 2.0  # all alike
        x[8, (y[8] + 1) % vocab] = torch.nan
        x[9, (y[9] + 1) % vocab] = torch.inf
        x[10] = torch.finfo(dtype).min  # masked with the type's lowest value
        x[11, : vocab // 2] = torch.finfo(dtype).min
        y[12] = vocab  # past the vocabulary
        x[13] = x[13].round()  # many equal ones
        x[14, :vocab] = torch.arange(vocab).to(dtype) / vocab * 8  # every one larger than those before
        x[15, :vocab] = -torch.arange(vocab).to(dtype) / vocab * 8
        x[16] = 0.0  # zeros of both signs are equal
        x[16, ::2] = -0.0
        x[17, :vocab] = -torch.inf  # fewer candidates than alternatives
        x[17, [0, vocab - 1]] = 1.0
        x[18, (y[18] + 1) % vocab] = 60.0  # nearly certain of another
        x[19] = torch.finfo(dtype).max / 8
    return x.to(dev())[:, :vocab], y.to(dev())


class Stats(R.Rows):
    """Rows with entropy, its bound, and the order of the logits."""

    def __init__(self, x, labels, tau, k):
        super().__init__(x, labels, tau)
        z = R.f64(x) / self.tau
        rows, vocab = z.shape
        self.bad = self.logp.isnan() | (self.d.isnan().any(1))
        fine = self.counts & ~self.bad
        z = torch.where(fine[:, None], z, torch.zeros_like(z))
        a = z.amax(1, keepdim=True) - z
        e = torch.exp(-a)
        total = e.sum(1)
        a = torch.where(e > 0, a, torch.zeros_like(a))
        mean = (e * a).sum(1) / total
        nan = torch.tensor(torch.nan, dtype=torch.float64)
        left = torch.where(fine, total.log() + mean, 0.0)
        self.entropy = torch.where(self.bad, nan, left)
        spread = (e * a * a).sum(1) / total
        self.entropy_tol = R.EPS * (3 * spread + 64 * mean + 32 + left)
        f = R.f64(x) + 0.0
        f = torch.where(fine[:, None], f, torch.full_like(f, -torch.inf))
        value, at = torch.sort(f, dim=1, descending=True, stable=True)
        value, at = value[:, :k], at[:, :k]
        if k > vocab:
            more = k - vocab
            value = torch.cat([value, torch.full((rows, more), -torch.inf, dtype=torch.float64)], 1)
            at = torch.cat([at, torch.zeros(rows, more, dtype=torch.int64)], 1)
        self.ids = torch.where(value > -torch.inf, at, torch.full_like(at, -1))
        # from the row's maximum: beside 1e38 even 64 bits hold no log(vocab)
        top = torch.where(value > -torch.inf, (value - value[:, :1]) / self.tau - total.log()[:, None], -torch.inf)
        self.tops = torch.where(self.bad[:, None], nan, top)


def check(x, y, tau, k, what):
    import hash_table_cache_amd as H

    want = Stats(x, y, tau, k)
    got = H.token_stats(x, y, k, temperature=tau)
    size = want.logp.abs().nan_to_num(0, 0, 0)
    R.assert_near(got.logp, want.logp, R.LOGP + size * R.EPS, f"logp {what}")
    R.assert_near(got.lse, want.lse, R.LOGP + want.lse.abs().nan_to_num(0, 0, 0) * R.EPS, f"lse {what}")
    R.assert_near(got.entropy, want.entropy, want.entropy_tol, f"entropy {what}")
    assert got.top_logp.shape == got.top_ids.shape == (x.shape[0], k)
    assert torch.equal(got.top_ids.cpu(), want.ids), f"ids {what}"
    # a log-probability is the difference of two numbers that 64 bits hold to 2^-52 of their size
    big = 2.0 ** -50 * (R.f64(x).nan_to_num(0, 0, 0).abs().amax(1) / want.tau)[:, None]
    tol = R.LOGP + want.tops.abs().nan_to_num(0, 0, 0) * R.EPS + torch.where(big > 1e-9, big, 0.0)
    R.assert_near(got.top_logp, want.tops, tol, f"tops {what}")
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_stats(vocab, dtype):
    for rows, pad, tau, k in ((1, 0, 1.0, 5), (37, 0, 1.0, 64), (37, 3, 0.75, 1), (20, 8, 4.0, 0), (70, 1, 1.0, 20)):
        x, y = make(rows, vocab, dtype, 100 + vocab, pad)
        check(x, y, tau, k, f"{rows} {pad}")


@pytest.mark.parametrize("rows,vocab,dtype,k", [(1, 300007, torch.bfloat16, 64), (3, 262144, torch.float32, 7),
                                                (66, 131072, torch.float16, 64), (4099, 333, torch.bfloat16, 33),
                                                (63, 16385, torch.float16, 2), (300, 70001, torch.bfloat16, 20)])
def test_stats_of_long_and_of_many_rows(rows, vocab, dtype, k):
    x, y = make(rows, vocab, dtype, 7)
    check(x, y, 1.0, k, "")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["up", "down", "alike", "steps", "zigzag"])
@pytest.mark.parametrize("rows,vocab", [(65, 20011), (2, 50021), (5, 700)])
def test_orders_that_many_pass(rows, vocab, order, dtype):
    """Rows in which far more than k elements come in reach of the list, and ties past it."""
    i = torch.arange(vocab, dtype=torch.float64)
    row = {"up": i / vocab * 16, "down": -i / vocab * 16, "alike": torch.full_like(i, -1.25),
           "steps": torch.floor(i / 1000) % 7, "zigzag": torch.where(i % 2 == 0, i, -i) / vocab * 16}[order]
    x = row.to(dtype).repeat(rows, 1).to(dev())
    x[1] = x[1].flip(0)
    y = torch.arange(rows, device=dev()) * 7
    for k in (1, 20, 64):
        check(x, y, 1.0, k, f"{order} {k}")


def backward_reference(x, y, tau, lse, h, g, ge):
    """The gradient from the operator's own lse and entropy, and its tolerance."""
    tau = float(torch.tensor(tau, dtype=torch.float32))
    z = (R.f64(x) / tau - R.f64(lse)[:, None]).clamp(min=-1e4)
    p = torch.exp(z)
    rows, vocab = z.shape
    at = torch.arange(rows), y.cpu().clamp(0, vocab - 1)
    g, ge, h = R.f64(g)[:, None], R.f64(ge)[:, None], R.f64(h)[:, None]
    d = -p * (g + ge * (z + h))
    d[at] = (g[:, 0] * -torch.expm1(z[at])) - (ge * p * (z + h))[at]
    size = p * (g.abs() + ge.abs() * (z + h).abs())
    size[at] = (g.abs()[:, 0] * -torch.expm1(z[at]).clamp(max=0)) + (ge.abs() * p * (z + h).abs())[at]
    apart = 4 * R.EPS * z.abs() + 2.0 ** -47 * R.f64(x).nan_to_num(0, 0, 0).abs() / tau
    tol = (size * (R.GRAD + 4 * R.EPS + 3 * R.EPS * z.abs()) + ge.abs() * p * apart) / tau
    tol = tol + 2.0 ** -126 * (g.abs() + ge.abs() * (z + h).abs()) / tau
    tol = tol + d.abs() / tau * R.half_step(x.dtype) + R.TINY[x.dtype]
    return d / tau, tol


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_backward(vocab, dtype):
    import hash_table_cache_amd as H

    for rows, pad, tau, inplace in ((1, 0, 1.0, False), (37, 0, 1.0, True), (37, 3, 0.75, False), (20, 1, 2.0, True)):
        x, y = make(rows, vocab, dtype, 300 + vocab, pad)
        # rows of the type's extreme values: their normalisers as floats do not tell the exponents
        for r in (10, 19):
            if rows > r:
                x[r] = torch.linspace(-2, 2, vocab).to(dtype)
        st = H.token_stats(x, y, temperature=tau)
        gen = torch.Generator().manual_seed(rows + vocab)
        g, ge = torch.randn(rows, generator=gen), torch.randn(rows, generator=gen)
        if rows > 1:
            g[0] = 0.0
            ge[15] = 0.0
            g[14] = ge[14] = 0.0
            g[8] = ge[8] = 0.0  # zeros, whatever the logits
        out = y < 0
        out |= st.lse == -torch.inf
        nan = st.logp.isnan().cpu() & ((g != 0) | (ge != 0))
        ref, tol = backward_reference(x, y, tau, st.lse, st.entropy, g, ge)
        ref[(out.cpu() | ((g == 0) & (ge == 0)))] = 0.0
        ref[nan] = torch.nan
        got = H.token_stats_backward(x, y, st.lse, st.entropy, g.to(dev()), ge.to(dev()), temperature=tau,
                                     grad_out=x if inplace else None)
        assert (got.data_ptr() == x.data_ptr()) == inplace
        R.assert_near(got, ref, tol.nan_to_num(0, 0, 0), f"grad {rows} {pad}")


def test_backward_of_one_kind():
    """Without one of the two gradients the other's alone; log-probability's is token_logprobs_backward's."""
    import hash_table_cache_amd as H

    x, y = make(40, 1003, torch.float32, 5)
    st = H.token_stats(x, y)
    g = torch.randn(40, device=dev())
    only = H.token_stats_backward(x, y, st.lse, grad_logp=g)
    assert torch.equal(only.nan_to_num(7.0), H.token_logprobs_backward(x, y, st.lse, g).nan_to_num(7.0))
    zero = torch.zeros_like(g)
    a = H.token_stats_backward(x, y, st.lse, st.entropy, grad_entropy=g)
    b = H.token_stats_backward(x, y, st.lse, st.entropy, zero, g)
    assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def test_backward_against_differences():
    import hash_table_cache_amd as H

    gen = torch.Generator().manual_seed(3)
    rows, vocab, tau, h = 6, 9, 0.8, 2.0 ** -5
    x = torch.randn(rows, vocab, generator=gen)
    y = torch.randint(0, vocab, (rows,), generator=gen).to(dev())
    g, ge = torch.randn(rows, generator=gen), torch.randn(rows, generator=gen)

    def value(x):
        st = H.token_stats(x.to(dev()), y, temperature=tau)
        return R.f64(st.logp) * g.double() + R.f64(st.entropy) * ge.double()

    st = H.token_stats(x.to(dev()), y, temperature=tau)
    got = H.token_stats_backward(x.to(dev()), y, st.lse, st.entropy, g.to(dev()), ge.to(dev()), temperature=tau)
    for v in range(vocab):
        step = torch.zeros(vocab)
        step[v] = h
        slope = (value(x + step) - value(x - step)) / (2 * h)
        # values to 64 eps of at most 8 each, differences to h^2 / 6 of a third derivative under 8 / tau^3
        tol = (g.abs() + ge.abs()).double() * (2 * 64 * 8 * R.EPS / (2 * h) + h * h / 6 * 8 / tau ** 3)
        R.assert_near(got[:, v], slope, tol, f"difference {v}")


def test_streams_graphs_and_memory():
    """Two calls at once on streams of their own, a captured call replayed on new logits, frames left alone."""
    import hash_table_cache_amd as H

    cases = [make(40, 40009, torch.bfloat16, 1), make(300, 5000, torch.bfloat16, 2)]
    want = [H.token_stats(x, y, 9) for x, y in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [H.token_stats(x, y, 9, stream=s) for (x, y), s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p.nan_to_num(7.0), q.nan_to_num(7.0)) for p, q in zip(a, b))

    wide = torch.full((40, 40009 + 64), 3.0, dtype=torch.bfloat16, device=dev())
    x, y = wide[:, :40009], cases[0][1]
    x.copy_(cases[0][0])
    g = torch.randn(40, device=dev())
    grad = torch.full_like(wide, 5.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st = H.token_stats(x, y, 9)
        H.token_stats_backward(x, y, st.lse, st.entropy, g, g, grad_out=grad[:, :40009])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = H.token_stats(x, y, 9)
        H.token_stats_backward(x, y, st.lse, st.entropy, g, g, grad_out=grad[:, :40009])
    for seed in (11, 12, 13):
        x.copy_(make(40, 40009, torch.bfloat16, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        eager = H.token_stats(x, y, 9)
        for p, q in zip(st, eager):
            assert torch.equal(p.nan_to_num(7.0), q.nan_to_num(7.0))
        back = H.token_stats_backward(x, y, eager.lse, eager.entropy, g, g)
        assert torch.equal(grad[:, :40009].nan_to_num(7.0), back.nan_to_num(7.0))
        assert bool((grad[:, 40009:] == 5.0).all())


def test_nothing_to_do():
    import hash_table_cache_amd as H

    x = torch.zeros(0, 50, device=dev())
    y = torch.zeros(0, dtype=torch.int64, device=dev())
    st = H.token_stats(x, y, 4)
    assert st.logp.shape == (0,) and st.top_ids.shape == (0, 4)
    assert H.token_stats_backward(x, y, st.lse, st.entropy, st.logp, st.logp).shape == (0, 50)


def test_refusals():
    import hash_table_cache_amd as H

    x, y = make(4, 100, torch.float32, 1)
    f = torch.zeros(4, device=dev())
    for k in (-1, 65):
        with pytest.raises(ValueError, match="outside 0 .. 64"):
            H.token_stats(x, y, k)
    with pytest.raises(TypeError):
        H.token_stats(x, y, 2.5)
    with pytest.raises(H.HkvError, match="temperature"):
        H.token_stats(x, y, 2, temperature=0.0)
    with pytest.raises(ValueError, match="grad_logp or grad_entropy"):
        H.token_stats_backward(x, y, f, f)
    with pytest.raises(ValueError, match="entropy is required"):
        H.token_stats_backward(x, y, f, grad_entropy=f)
    with pytest.raises(ValueError, match="lse has shape"):
        H.token_stats_backward(x, y, f[:3], f, f, f)
    with pytest.raises(TypeError, match="grad_entropy"):
        H.token_stats_backward(x, y, f, f, f, f.double())
    with pytest.raises(H.HkvError, match="overlaps"):
        wide = torch.zeros(4, 200, device=dev())
        H.token_stats_backward(wide[:, :100], y, f, f, f, f, grad_out=wide[:, 50:150])
