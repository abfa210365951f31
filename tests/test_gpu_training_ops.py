"""The training operators against their formulas in 64 bits: log-probabilities
forward and backward, preference and policy losses, gradient clipping."""

import math

import pytest
import torch

import training_reference as R
from conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# one element, less than a vector, around vectors, waves and workgroups, odd ones
VOCABS = [1, 2, 7, 8, 9, 64, 100, 511, 513, 1000, 2049, 8192, 8195, 40009]


def dev():
    return torch.device("cuda", 0)


def make(rows, vocab, dtype, seed, pad=0, special=True, lowest=1.0):
    """Logits with the rows that go wrong among ordinary ones, and labels."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab + pad, generator=gen) * 3.0
    x = x.to(dtype)
    y = torch.randint(0, vocab, (rows,), generator=gen)
    x[torch.arange(rows), y] += 3.0
    if special and rows >= 16:
        x[1] = -torch.inf  # nothing left
        x[2, :vocab] = -torch.inf  # one candidate left, the label
        x[2, y[2]] = 1.5
        x[3, y[3]] = -torch.inf  # the label masked beside others
        y[4] = -100  # left out, with NaN among its logits
        x[4, 0] = torch.nan
        x[5, y[5]] = 40.0  # nearly certain
        x[6, : vocab // 2] = -torch.inf  # half masked
        x[7, :] = 2.0  # all alike
        x[8, (y[8] + 1) % vocab] = torch.nan
        x[9, (y[9] + 1) % vocab] = torch.inf
        x[10, :] = torch.finfo(dtype).min * lowest  # masked with the type's lowest value
        x[11, : vocab // 2] = torch.finfo(dtype).min
        y[12] = -1
        y[13] = vocab  # past the vocabulary
        x[14] = -torch.inf  # nothing left, and no label
        y[14] = -5
        x[15, y[15]] = torch.inf
    x = x.to(dev())[:, :vocab]
    return x, y.to(dev())


def grad_tolerance(rows, g, dtype, delta_g):
    """Elementwise: relative error of p, error of the coefficient, rounding."""
    ref = rows.grad(g).abs()
    # an infinite or NaN coefficient has no tolerance
    return ref * (R.GRAD + R.half_step(dtype)) + rows.d.abs() * (delta_g / rows.tau)[:, None] + R.TINY[dtype]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprobs(vocab, dtype):
    import hash_table_cache_amd as H

    for rows, pad, tau in ((1, 0, 1.0), (37, 0, 1.0), (37, 3, 0.7), (16, 8, 4.0)):
        x, y = make(rows, vocab, dtype, 100 + vocab, pad)
        want = R.Rows(x, y, tau)
        logp, lse = H.token_logprobs(x, y, temperature=tau)
        R.assert_near(logp, want.logp, R.LOGP + want.logp.abs().nan_to_num(0, 0, 0) * R.EPS, f"logp {rows} {pad}")
        R.assert_near(lse, want.lse, R.LOGP + want.lse.abs().nan_to_num(0, 0, 0) * R.EPS, f"lse {rows} {pad}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_backward(vocab, dtype):
    import hash_table_cache_amd as H

    for rows, pad, tau, inplace in ((1, 0, 1.0, False), (37, 0, 1.0, True), (37, 3, 0.75, False), (16, 1, 2.0, True)):
        # a row of float32's lowest value has a normaliser past its range where the temperature is under 1
        x, y = make(rows, vocab, dtype, 200 + vocab, pad, lowest=0.5)
        want = R.Rows(x, y, tau)
        lse = want.lse.float()
        g = torch.linspace(-2.0, 3.0, rows)
        if rows > 1:
            g[rows // 2] = 0.0
        # the operator's own lse, rounded to 32 bits, is its input: p = exp(x / tau - lse)
        z = R.f64(x) / want.tau - lse.double()[:, None]
        d = -torch.exp(z)
        at = y.cpu().clamp(0, vocab - 1)
        d[torch.arange(rows), at] = -torch.expm1(z[torch.arange(rows), at])
        nan = want.d.isnan().all(1)
        d = torch.where(nan[:, None], torch.nan, torch.where(want.counts[:, None], d, 0.0))
        want.d = d
        grad = H.token_logprobs_backward(x, y, lse.to(dev()), g.to(dev()), temperature=tau,
                                         grad_out=x if inplace else None)
        assert (grad.data_ptr() == x.data_ptr()) == inplace
        ref = want.grad(g.double())
        tol = ref.abs() * (R.GRAD + R.half_step(dtype)) + R.TINY[dtype]
        # where lse is past 2^30, x / tau - lse is known neither in 32 bits nor in 64 (its rounding alone moves the
        # exponent by units): there only that it is held to 1
        lost = lse.abs() > 2.0 ** 30
        lost &= lse.isfinite()
        most = (g.double().abs() / want.tau * (math.e + R.half_step(dtype) * 4))[:, None] + R.TINY[dtype]
        assert bool((R.f64(grad).abs() <= most)[lost].all())
        R.assert_near(grad[~lost.to(dev())], ref[~lost], tol[~lost].nan_to_num(0, 0, 0), f"grad {rows} {pad}")


def sequences(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int64)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 9, 100, 1000, 8195])
@pytest.mark.parametrize("lengths,before,after", [([3, 4], 0, 0), ([0, 5, 1, 0], 2, 3), ([17, 9, 1, 1, 0, 0, 40, 300], 0, 1)])
def test_preference(lengths, before, after, vocab, dtype):
    import hash_table_cache_amd as H

    rows = before + sum(lengths) + after
    cu = sequences(lengths) + before
    for special, smoothing, tau, with_ref in ((False, 0.0, 1.0, True), (False, 0.1, 0.7, False), (True, 0.05, 1.0, True)):
        x, y = make(rows, vocab, dtype, 300 + vocab, 0, special=False)
        if special:  # left out, nothing left, half masked
            y[rows // 2] = -100
            x[rows // 3] = -torch.inf
            x[rows // 4, : vocab // 2] = -torch.inf
            y[rows // 4] = vocab - 1
        want = R.Rows(x, y, tau)
        ref = (want.logp + 0.3 * torch.randn(rows, generator=torch.Generator().manual_seed(5)).double()).float()
        beta, scale = 0.2, 16.0
        loss, losses, rewards, g = R.preference(want, cu, ref if with_ref else None, beta, smoothing, scale)
        got = H.preference_loss(x, y, cu.to(dev()), ref.to(dev()) if with_ref else None, beta=beta,
                                label_smoothing=smoothing, temperature=tau, grad_scale=scale)
        n = torch.tensor(lengths, dtype=torch.float64)
        d_reward = beta * n * R.LOGP
        d_margin = d_reward[0::2] + d_reward[1::2]
        R.assert_near(got.logp, want.logp, R.LOGP + want.logp.abs() * R.EPS, "logp")
        R.assert_near(got.rewards, rewards, d_reward + rewards.abs() * R.EPS, "rewards")
        R.assert_near(got.losses, losses, d_margin + losses.abs() * R.EPS, "losses")
        R.assert_near(got.loss, loss, d_margin.max() + loss.abs() * R.EPS, "loss")
        pair_of = torch.zeros(rows, dtype=torch.int64)
        for s in range(len(lengths)):
            pair_of[cu[s]:cu[s + 1]] = s // 2
        # sigma' <= 1/4
        delta = scale * beta / (len(lengths) // 2) * d_margin[pair_of] / 4 + g.abs() * 4 * R.EPS
        R.assert_near(got.grad, want.grad(g), grad_tolerance(want, g, dtype, delta), "grad")
        plain = H.preference_loss(x, y, cu.to(dev()), ref.to(dev()) if with_ref else None, beta=beta,
                                  label_smoothing=smoothing, temperature=tau, with_grad=False)
        assert plain.grad is None and torch.equal(plain.loss, got.loss) and torch.equal(plain.rewards, got.rewards)


def test_preference_without_pairs_or_rows():
    import hash_table_cache_amd as H

    x, y = make(5, 30, torch.float32, 1)
    got = H.preference_loss(x, y, torch.zeros(1, dtype=torch.int64, device=dev()))
    assert float(got.loss) == 0.0 and bool((got.grad == 0).all()) and got.losses.numel() == 0
    got = H.preference_loss(x[:0], y[:0], torch.zeros(3, dtype=torch.int64, device=dev()))
    assert float(got.loss) == pytest.approx(math.log(2.0), abs=1e-7) and got.rewards.tolist() == [0.0, 0.0]


def test_preference_offsets_are_clamped():
    """Offsets outside the rows or going back read and write nothing outside."""
    import hash_table_cache_amd as H

    x, y = make(12, 50, torch.float32, 2)
    good = H.preference_loss(x, y, torch.tensor([0, 4, 12], device=dev()))
    got = H.preference_loss(x, y, torch.tensor([-7, 4, 1 << 40], device=dev()))
    assert torch.equal(got.loss, good.loss) and torch.equal(got.grad, good.grad)
    got = H.preference_loss(x, y, torch.tensor([5, 2, 2], device=dev()))  # the first ends before it begins
    assert float(got.loss) == pytest.approx(math.log(2.0), abs=1e-7) and bool((got.grad == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy(vocab, dtype):
    import hash_table_cache_amd as H

    for rows, pad, tau, kl_coef, inplace in ((1, 0, 1.0, 0.0, False), (41, 0, 1.0, 0.1, True), (41, 5, 0.7, 0.0, False),
                                             (41, 0, 1.5, 0.2, False)):
        x, y = make(rows, vocab, dtype, 400 + vocab, pad)
        want = R.Rows(x, y, tau)
        gen = torch.Generator().manual_seed(9)
        low, high = 0.2, 0.3
        d = 0.4 * torch.randn(rows, generator=gen).double()
        for border in (math.log(1 - low), math.log(1 + high)):  # none on a bound
            d = torch.where((d - border).abs() < 1e-3, d + 2e-3, d)
        base = want.logp.nan_to_num(0.0, 0.0, -3.0)
        old = (base - d).float()
        ref = (base + 0.2 * torch.randn(rows, generator=gen).double()).float() if kl_coef else None
        adv = torch.randn(rows, generator=gen)
        w = torch.rand(rows, generator=gen)
        w[rows // 2] = 0.0
        scale = 32.0
        total, loss, kl, g = R.policy(want, old, adv, w, ref, low, high, kl_coef, scale)
        got = H.policy_loss(x, y, old.to(dev()), adv.to(dev()), w.to(dev()), None if ref is None else ref.to(dev()),
                            clip_low=low, clip_high=high, kl_coef=kl_coef, temperature=tau, grad_scale=scale,
                            grad_out=x if inplace else None)
        assert (got.grad.data_ptr() == x.data_ptr()) == inplace
        # one unit of logp moves r A by r A and the divergence by e^d - 1
        r = torch.exp(want.logp - old.double()).nan_to_num(0, 0, 0)
        e = torch.zeros(rows).double() if ref is None else torch.exp(ref.double() - want.logp).nan_to_num(0, 0, 0)
        slope = (r * adv.double()).abs() + kl_coef * (e + 1)
        tol = slope * R.LOGP + loss.abs().nan_to_num(0, 0, 0) * R.EPS
        R.assert_near(got.logp, want.logp, R.LOGP + want.logp.abs().nan_to_num(0, 0, 0) * R.EPS, "logp")
        R.assert_near(got.token_loss, loss, tol, "token_loss")
        R.assert_near(got.kl, kl, (e + 1) * R.LOGP + kl.abs().nan_to_num(0, 0, 0) * R.EPS, "kl")
        R.assert_near(got.loss, total, (w.double() * (tol + loss.abs().nan_to_num(0, 0, 0) * R.EPS)).sum() + total.abs() * R.EPS, "loss")
        delta = slope * R.LOGP * w.double() * scale + g.abs().nan_to_num(0, 0, 0) * 4 * R.EPS
        tol = grad_tolerance(want, g, dtype, delta)
        R.assert_near(got.grad, want.grad(g), tol.nan_to_num(0, 0, 0), "grad")


@pytest.mark.parametrize("clipped", [False, True])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [16384], [16385, 3, 70000], [7] * 250, [100003, 1, 0, 333]])
def test_clip(sizes, clipped):
    import hash_table_cache_amd as H

    gen = torch.Generator().manual_seed(sum(sizes))
    flats, grads = [], []
    for i, n in enumerate(sizes):  # views that begin at any element
        flat = torch.randn(n + i % 5, generator=gen).to(TYPES[i % 3]).to(dev())
        flats.append(flat)
        grads.append(flat[i % 5:])
    before = [R.f64(g) for g in grads]
    norm = math.sqrt(sum(float(g.square().sum()) for g in before))
    bound = norm * (0.25 if clipped else 1.5)
    bound32 = float(torch.tensor(bound, dtype=torch.float32))
    coef = min(1.0, bound32 / norm) if norm else 1.0
    outs = [torch.full_like(g, torch.nan) for g in grads]
    heads = [R.f64(f[:i % 5]) for i, f in enumerate(flats)]
    got = H.clip_grad_norm(grads, bound, out=outs)
    R.assert_near(got, torch.tensor(norm, dtype=torch.float64), 2 * norm * R.EPS, "norm")
    for g, b, o in zip(grads, before, outs):
        assert torch.equal(R.f64(g), b)  # out of place: untouched
        R.assert_near(o, b * coef, (b * coef).abs() * (2 * R.EPS + R.half_step(o.dtype)) + R.TINY[o.dtype], "out")
    got = H.clip_grad_norm(grads, bound)
    for f, h, g, b, o in zip(flats, heads, grads, before, outs):
        assert torch.equal(R.f64(f[:h.numel()]), h)
        assert torch.equal(g, o)  # in place gives the same bits


def test_clip_range_and_nonfinite():
    import hash_table_cache_amd as H

    def clip(vals, bound, dtype=torch.float32):
        t = torch.tensor(vals, dtype=dtype, device=dev())
        return float(H.clip_grad_norm([t], bound)), t.double().cpu().tolist()

    # squares past the range of 32 bits on both sides
    n, t = clip([3e30, 4e30], 1.0)
    assert n == pytest.approx(5e30, rel=1e-6) and t == pytest.approx([0.6, 0.8], rel=1e-6)
    n, t = clip([3e-30, 4e-30], 1e-30)
    assert n == pytest.approx(5e-30, rel=1e-6) and t == pytest.approx([6e-31, 8e-31], rel=1e-6)
    assert clip([0.0, 0.0], 0.0) == (0.0, [0.0, 0.0])
    assert clip([3.0, 4.0], 0.0) == (5.0, [0.0, 0.0])
    assert clip([3.0, 4.0], math.inf) == (5.0, [3.0, 4.0])
    n, t = clip([math.inf, 1.0], 1.0)
    assert n == math.inf and math.isnan(t[0]) and t[1] == 0.0
    n, t = clip([math.nan, 1.0], 1.0)
    assert math.isnan(n) and all(math.isnan(v) for v in t)


def test_clip_axes_in_any_order():
    import hash_table_cache_amd as H

    g = torch.randn(33, 65, device=dev()).t()
    want = g.clone()
    n = H.clip_grad_norm([g], 0.5)
    assert torch.allclose(g, want * (0.5 / float(n)), rtol=1e-6)


def test_past_32_bits():
    """Rows whose elements lie past 2^32 elements and bytes from the first."""
    import hash_table_cache_amd as H

    vocab, rows = 1 << 18, (1 << 14) + 3
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device=dev())
    pick = [0, 1, (1 << 13) - 1, 1 << 13, (1 << 14) - 1, 1 << 14, rows - 1]
    gen = torch.Generator(device=dev()).manual_seed(3)
    x[pick] = torch.randn(len(pick), vocab, dtype=torch.bfloat16, device=dev(), generator=gen)
    y = torch.full((rows,), -1, dtype=torch.int64, device=dev())
    y[pick] = torch.tensor([5, 77, 1000, vocab - 1, 3, vocab // 2, 9], device=dev())
    one = torch.ones(rows, device=dev())
    zero = torch.zeros(rows, device=dev())
    kept = x[pick].clone()
    want = R.Rows(kept, y[pick], 1.0)
    got = H.policy_loss(x, y, zero - 12.0, one, one, clip_high=1e30, grad_out=x)
    R.assert_near(got.logp[pick], want.logp, R.LOGP + want.logp.abs() * R.EPS, "logp")
    g = -torch.exp(want.logp + 12.0)
    tol = grad_tolerance(want, g, torch.bfloat16, g.abs() * R.LOGP)
    R.assert_near(got.grad[pick], want.grad(g), tol, "grad")
    rest = torch.ones(rows, dtype=torch.bool)
    rest[pick] = False
    assert not bool(x[rest.to(dev())][::97].any())


def test_gradient_against_differences():
    """Central differences of the losses (float32 logits, small steps in
    float64 through the reference) along random directions."""
    import hash_table_cache_amd as H

    rows, vocab = 12, 40
    x, y = make(rows, vocab, torch.float32, 77, special=False)
    cu = torch.tensor([0, 5, 7, 8, 12])
    ref = torch.randn(rows, generator=torch.Generator().manual_seed(1)) * 0.3 - 3.0
    adv = torch.randn(rows, generator=torch.Generator().manual_seed(2))
    w = torch.rand(rows, generator=torch.Generator().manual_seed(3))
    old = (R.Rows(x, y, 0.8).logp + 0.05).float()
    pref = H.preference_loss(x, y, cu.to(dev()), ref.to(dev()), beta=0.5, label_smoothing=0.1, temperature=0.8)
    pol = H.policy_loss(x, y, old.to(dev()), adv.to(dev()), w.to(dev()), ref.to(dev()), kl_coef=0.3, temperature=0.8)
    for seed in range(4):
        v = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(50 + seed)).double()
        h = 1e-5

        def at(step):
            r = R.Rows(R.f64(x) + step * v, y, 0.8)
            return (R.preference(r, cu, ref, 0.5, 0.1, 1.0)[0], R.policy(r, old, adv, w, ref, 0.2, 0.2, 0.3, 1.0)[0])

        up, down = at(h), at(-h)
        for k, got in enumerate((pref.grad, pol.grad)):
            diff = float(up[k] - down[k]) / (2 * h)
            assert float((R.f64(got) * v).sum()) == pytest.approx(diff, rel=1e-5, abs=1e-6)


def test_streams_and_graph():
    """Calls on a stream of their own, and captured: every replay, with other
    work and new inputs in between, equals the eager result."""
    import hash_table_cache_amd as H

    rows, vocab = 40, 5003
    x, y = make(rows, vocab, torch.bfloat16, 5, special=False)
    cu = torch.tensor([0, 9, 20, 31, 40], device=dev())
    old = torch.full((rows,), -4.0, device=dev())
    ones = torch.ones(rows, device=dev())
    grads = [torch.randn(n, device=dev()) for n in (100, 20000, 3)]
    outs = [torch.empty_like(g) for g in grads]

    def all_ops():
        logp, lse = H.token_logprobs(x, y)
        back = H.token_logprobs_backward(x, y, lse, ones)
        a = H.preference_loss(x, y, cu, old)
        b = H.policy_loss(x, y, old, ones, ones, old, kl_coef=0.1)
        n = H.clip_grad_norm(grads, 1.0, out=outs)
        return [logp, lse, back, *a, *b, n]

    eager = [t.clone() for t in all_ops()] + [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = H.preference_loss(x, y, cu, old, stream=side)
    n = H.clip_grad_norm(grads, 1.0, out=outs, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(a.grad, eager[7]) and torch.equal(n, eager[13])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_ops()
    for turn in range(4):
        x.copy_(torch.randn(rows, vocab, device=dev(), generator=torch.Generator(device=dev()).manual_seed(turn)))
        for g in grads:
            g.normal_()
        torch.cuda.synchronize()
        want = [t.clone() for t in all_ops()] + [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (h, w) in enumerate(zip([*held, *outs], want)):
            assert torch.equal(h, w), (turn, i)
        torch.randn(1000, 1000, device=dev()) @ torch.randn(1000, 1000, device=dev())
        torch.cuda.synchronize()


def test_repeats_are_bitwise_equal():
    import hash_table_cache_amd as H

    x, y = make(200, 4099, torch.bfloat16, 6, special=False)
    cu = torch.tensor([0, 100, 200], device=dev())
    first = H.preference_loss(x, y, cu)
    for _ in range(3):
        again = H.preference_loss(x, y, cu)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [5, 300, 1025, 4999, 20001])
@pytest.mark.parametrize("shift", [0, 1, 3, 64])
def test_nothing_is_written_outside_the_rows(vocab, shift, dtype):
    """Logits and gradient inside wider arrays, at every kind of alignment and
    of different ones: what lies around the rows stays as it was."""
    import hash_table_cache_amd as H

    rows, wide = 9, vocab + 70
    gen = torch.Generator().manual_seed(shift)
    whole = torch.randn(rows, wide, generator=gen).to(dtype).to(dev())
    x = whole[:, shift:shift + vocab]
    y = torch.randint(0, vocab, (rows,), generator=gen).to(dev())
    y[4] = -1
    want = R.Rows(x, y, 1.0)
    f = (want.logp + 0.05).float().to(dev())
    ones = torch.ones(rows, device=dev())
    cu = torch.tensor([0, 4, 9], device=dev())
    for call in (lambda o: H.token_logprobs_backward(x, y, want.lse.float().to(dev()), ones, grad_out=o),
                 lambda o: H.preference_loss(x, y, cu, f, grad_out=o).grad,
                 lambda o: H.policy_loss(x, y, f, ones, ones, grad_out=o).grad):
        plain = call(None)
        frame = torch.full((rows + 2, wide + 1), 7.0, dtype=dtype, device=dev())
        inner = frame[1:-1, 2 + shift // 2:2 + shift // 2 + vocab]
        call(inner)
        # another alignment sums a row in another order: both results within their bound of the formula
        near = 2 * (R.GRAD + R.half_step(dtype)) * R.f64(plain).abs() + R.TINY[dtype]
        R.assert_near(inner, R.f64(plain), near, "grad")
        inner.fill_(7.0)
        assert bool((frame == 7.0).all())
    before = whole.clone()
    H.policy_loss(x, y, f, ones, ones, grad_out=x)  # in place
    assert torch.equal(whole[:, :shift], before[:, :shift])
    assert torch.equal(whole[:, shift + vocab:], before[:, shift + vocab:])


def test_refusals_on_the_gpu():
    import hash_table_cache_amd as H

    x, y = make(6, 40, torch.float32, 3, special=False)
    f = torch.zeros(6, device=dev())
    cu = torch.tensor([0, 3, 6], device=dev())
    with pytest.raises(TypeError, match="labels"):
        H.token_logprobs(x, y.int())
    with pytest.raises(ValueError, match="labels"):
        H.token_logprobs(x, y[:5])
    with pytest.raises(ValueError, match="labels"):
        H.token_logprobs(x, y.cpu())
    with pytest.raises(ValueError, match="next to each other"):
        H.token_logprobs(x.t().contiguous().t(), y)
    with pytest.raises(ValueError, match="overlap"):
        H.token_logprobs(x[:1].expand(6, 40), y)
    with pytest.raises(ValueError, match="cu_seqlens"):
        H.preference_loss(x, y, cu[:2], f)
    with pytest.raises(ValueError, match="kl_coef"):
        H.policy_loss(x, y, f, f, f, kl_coef=0.1)
    with pytest.raises(ValueError, match="grad_out"):
        H.policy_loss(x, y, f, f, f, grad_out=torch.empty(6, 41, device=dev()))
    wide = torch.zeros(7, 40, device=dev())
    with pytest.raises(H.HkvError, match="overlaps"):
        H.policy_loss(wide[:6], y, f, f, f, grad_out=wide[1:])
    with pytest.raises(H.HkvError, match="temperature"):
        H.token_logprobs(x, y, temperature=0.0)
    with pytest.raises(H.HkvError, match="max_norm"):
        H.clip_grad_norm([f], -1.0)
    g = torch.ones(100, device=dev())
    with pytest.raises(H.HkvError, match="overlap"):
        H.clip_grad_norm([g, g], 1.0)
    with pytest.raises(H.HkvError, match="overlap"):
        H.clip_grad_norm([g[:60], g[50:]], 1.0)
    with pytest.raises(H.HkvError, match="overlap"):
        H.clip_grad_norm([g[:60]], 1.0, out=[g[10:70]])
    with pytest.raises(ValueError, match="stretch"):
        H.clip_grad_norm([g.view(10, 10)[:, :5]], 1.0)
    with pytest.raises(H.HkvError, match="pageable"):
        H.clip_grad_norm([g, torch.ones(5)], 1.0)
    with pytest.raises(ValueError, match="out"):
        H.clip_grad_norm([g], 1.0, out=[g.half()])
    with pytest.raises(ValueError, match="tensors in out"):
        H.clip_grad_norm([g], 1.0, out=[])
    assert bool((g == 1.0).all())  # no refused call has written


def test_lists_longer_than_a_launch_holds():
    """More tensors than the kernels' arguments or their shared memory hold."""
    import hash_table_cache_amd as H

    for n in (140, 141, 281, 2049, 5000):
        sizes = [1 + (i * 37) % 90 for i in range(n)]
        flat = torch.randn(sum(sizes), device=dev())
        want = f_norm = float(R.f64(flat).norm())
        out = torch.zeros_like(flat)
        got = H.clip_grad_norm(flat.split(sizes), 0.5 * want, out=out.split(sizes))
        assert float(got) == pytest.approx(f_norm, rel=1e-6)
        coef = float(torch.tensor(0.5 * want, dtype=torch.float32)) / f_norm
        R.assert_near(out, R.f64(flat) * coef, R.f64(out).abs() * 4 * R.EPS + 1e-30, f"out {n}")


def test_example_learns():
    import importlib.util
    import pathlib

    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "online_feedback.py"
    spec = importlib.util.spec_from_file_location("online_feedback", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    preference, policy = example.train(steps=40)
    assert preference[0] == pytest.approx(math.log(2.0), rel=1e-3)  # the model is its own reference at first
    assert preference[-1] < 0.8 * preference[0]
    assert all(math.isfinite(v) for v in preference + policy)


def test_policy_far_from_the_old_policy():
    """Ratios and divergences past a float's range, on both sides, and an advantage of 0."""
    import hash_table_cache_amd as H

    shifts = [300.0, 175.0, 100.0, 85.0, 60.0, 0.4999, 0.5001, -0.5001, 0.0, -60.0, -150.0, -300.0]
    rows = 3 * len(shifts)
    x, y = make(rows, 33, torch.float32, 8, special=False)
    want = R.Rows(x, y, 1.0)
    d = torch.tensor(shifts * 3, dtype=torch.float64)
    old, ref = (want.logp - d).float(), (want.logp + d).float()
    adv = torch.tensor([1.0] * len(shifts) + [-1.0] * len(shifts) + [0.0] * len(shifts))
    w = torch.full((rows,), 1e-3)
    for kl_coef, ref_ in ((0.0, None), (0.1, ref)):
        total, loss, kl, g = R.policy(want, old, adv, w, ref_, 0.2, 0.2, kl_coef, 1.0)
        got = H.policy_loss(x, y, old.to(dev()), adv.to(dev()), w.to(dev()), None if ref_ is None else ref_.to(dev()),
                            kl_coef=kl_coef)
        r = torch.exp(want.logp - old.double())
        e = torch.exp(ref_.double() - want.logp) if kl_coef else torch.zeros_like(r)
        slope = (r * adv.double()).abs() + kl_coef * (e + 1)
        R.assert_near(got.token_loss, loss, slope * R.LOGP + loss.abs() * R.EPS + 1e-37, "token_loss")
        R.assert_near(got.kl, kl, (e + 1) * R.LOGP + kl.abs() * R.EPS, "kl")
        delta = slope * R.LOGP * w.double() + g.abs() * 4 * R.EPS
        ref_grad = want.grad(g)
        tol = grad_tolerance(want, g, torch.float32, delta)
        fine = ref_grad.abs().amax(1) < 1e37  # an infinite coefficient times a small probability is infinite, not small
        R.assert_near(got.grad[fine.to(dev())], ref_grad[fine], tol[fine] + 1e-37, "grad")


# rows enough that every length goes to the teams of many rows: vectors a row up to 4096, 8192, 12288 and more
@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 9001), (torch.float32, 32003), (torch.float32, 33001),
                                         (torch.float32, 60007), (torch.bfloat16, 20001), (torch.bfloat16, 50021),
                                         (torch.bfloat16, 66003), (torch.bfloat16, 100003), (torch.float16, 66003),
                                         (torch.float16, 1 << 17)])
def test_many_rows(dtype, vocab):
    import hash_table_cache_amd as H

    rows = 259
    x, y = make(rows, vocab, dtype, 700 + vocab % 1000, pad=5)
    x[20, :] = -torch.inf  # one candidate, in the last place; the first; a huge gap
    x[20, vocab - 1], y[20] = 1.0, vocab - 1
    y[21] = 0
    x[22, vocab // 2], y[22] = 60000.0, vocab // 2
    x[23, vocab // 3], y[23] = 60000.0, vocab // 2
    want = R.Rows(x, y, 0.75)
    gen = torch.Generator().manual_seed(4)
    base = want.logp.nan_to_num(0.0, 0.0, -3.0)
    old = (base + 0.05).float()
    adv, w = torch.randn(rows, generator=gen), torch.rand(rows, generator=gen)
    logp, lse = H.token_logprobs(x, y, temperature=0.75)
    R.assert_near(logp, want.logp, R.LOGP + want.logp.abs().nan_to_num(0, 0, 0) * R.EPS, "logp")
    total, loss, kl, g = R.policy(want, old, adv, w, None, 0.2, 0.2, 0.0, 256.0)
    slope = (torch.exp(want.logp - old.double()).nan_to_num(0, 0, 0) * adv.double()).abs()
    delta = slope * R.LOGP * w.double() * 256.0 + g.abs().nan_to_num(0, 0, 0) * 4 * R.EPS
    tol = grad_tolerance(want, g, dtype, delta).nan_to_num(0, 0, 0)
    for out in (None, x):
        got = H.policy_loss(x, y, old.to(dev()), adv.to(dev()), w.to(dev()), temperature=0.75, grad_scale=256.0,
                            grad_out=out)
        R.assert_near(got.logp, want.logp, R.LOGP + want.logp.abs().nan_to_num(0, 0, 0) * R.EPS, "policy logp")
        R.assert_near(got.grad, want.grad(g), tol, "grad")


def test_policy_loss_that_cancels():
    """Terms of both signs whose sum is a thousandth of their size."""
    import hash_table_cache_amd as H

    rows, vocab = 2000, 50
    x, y = make(rows, vocab, torch.float32, 21, special=False)
    want = R.Rows(x, y, 1.0)
    old = want.logp.float()
    adv = torch.randn(rows, generator=torch.Generator().manual_seed(2))
    adv -= adv.mean() - 1e-3
    w = torch.full((rows,), 1.0 / rows)
    total, loss, _, _ = R.policy(want, old, adv, w, None, 0.2, 0.2, 0.0, 1.0)
    got = H.policy_loss(x, y, old.to(dev()), adv.to(dev()), w.to(dev()))
    # each term's error is its logp's, at most 32 eps but of either sign: a random walk of 2000 steps, sixfold
    walk = 6 * math.sqrt(rows) * float(adv.abs().max()) * 4 * R.EPS / rows
    assert float(got.loss) == pytest.approx(float(total), abs=walk)


# rows enough for the small teams: up to 64, 128, 256, 512, 1024, 2048 and 4096 vectors a row
@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 8), (torch.bfloat16, 509), (torch.float16, 1003),
                                         (torch.bfloat16, 2001), (torch.float32, 2047), (torch.bfloat16, 4099),
                                         (torch.bfloat16, 8111), (torch.float32, 7001), (torch.float16, 16001),
                                         (torch.bfloat16, 30011)])
def test_thousands_of_rows(dtype, vocab):
    import hash_table_cache_amd as H

    rows = 4099
    gen = torch.Generator(device=dev()).manual_seed(vocab)
    x = torch.randn(rows, vocab, device=dev(), generator=gen).mul_(3.0).to(dtype)
    y = torch.randint(0, vocab, (rows,), device=dev(), generator=gen)
    some, labels = make(48, vocab, dtype, 900 + vocab)
    pick = torch.cat([torch.arange(0, 32), torch.arange(2050, 2058), torch.arange(rows - 8, rows)])
    x[pick.to(dev())], y[pick.to(dev())] = some, labels
    want = R.Rows(some, labels, 1.25)
    logp, lse = H.token_logprobs(x, y, temperature=1.25)
    R.assert_near(logp[pick], want.logp, R.LOGP + want.logp.abs().nan_to_num(0, 0, 0) * R.EPS, "logp")
    near = R.LOGP + want.logp.abs().nan_to_num(0, 0, 0) * R.EPS
    ones = torch.ones(rows, device=dev())
    old = logp.nan_to_num(0.0, 0.0, -3.0) - 0.05
    adv = torch.randn(rows, device=dev(), generator=gen)
    got = H.policy_loss(x, y, old, adv, ones, temperature=1.25, grad_scale=8.0)
    total, loss, kl, g = R.policy(want, old[pick], adv[pick], ones[pick], None, 0.2, 0.2, 0.0, 8.0)
    slope = (torch.exp(want.logp - R.f64(old[pick])).nan_to_num(0, 0, 0) * R.f64(adv[pick])).abs()
    delta = slope * R.LOGP * 8.0 + g.abs().nan_to_num(0, 0, 0) * 4 * R.EPS
    R.assert_near(got.logp[pick], want.logp, near, "policy logp")
    R.assert_near(got.grad[pick], want.grad(g), grad_tolerance(want, g, dtype, delta).nan_to_num(0, 0, 0), "policy grad")
    # one pair of all rows without the special ones, whose NaN would be everyone's
    y2 = y.clone()
    y2[pick.to(dev())] = -1
    y2[40:60] = torch.arange(20, device=dev()) % vocab
    pref = H.preference_loss(x, y2, torch.tensor([0, 2000, rows], device=dev()), temperature=1.25, grad_scale=8.0)
    sub = torch.arange(40, 60)
    want = R.Rows(x[40:60], y2[40:60], 1.25)
    R.assert_near(pref.logp[sub], want.logp, R.LOGP + want.logp.abs() * R.EPS, "pair logp")
    reward = R.f64(pref.rewards)
    c = 0.1 * (torch.sigmoid(reward[0] - reward[1]) - 1) * 8.0
    g = torch.full((20,), float(c), dtype=torch.float64)
    # the margin from the float32 rewards is off by an eps of each, sigma by a quarter of that
    delta = 0.1 * 8.0 * reward.abs().sum() * R.EPS / 4 + g.abs() * 4 * R.EPS
    R.assert_near(pref.grad[sub], want.grad(g), grad_tolerance(want, g, dtype, delta), "pair grad")
    assert not bool(pref.grad[pick].any())
    back = H.token_logprobs_backward(x[40:60], y2[40:60], want.lse.float().to(dev()), g.float().to(dev()), temperature=1.25)
    assert back.shape == (20, vocab)


# few rows so long that workgroups share them: an even cut, a short last part, more than 64 parts' worth
@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 65541), (torch.float32, 600011), (torch.bfloat16, 131081),
                                         (torch.float16, 262144), (torch.bfloat16, 1500007)])
def test_few_long_rows(dtype, vocab):
    import hash_table_cache_amd as H

    rows = 20
    x, y = make(rows, vocab, dtype, 800, pad=3)
    x[16, :] = -torch.inf  # a single candidate at either end, and in the middle
    x[16, vocab - 1], y[16] = 1.0, vocab - 1
    x[17, :] = -torch.inf
    x[17, 0], y[17] = 1.0, 0
    x[18, :] = -torch.inf
    x[18, vocab // 2], x[18, vocab // 3], y[18] = 1.0, 2.0, vocab // 3
    want = R.Rows(x, y, 0.75)
    near = R.LOGP + want.logp.abs().nan_to_num(0, 0, 0) * R.EPS
    logp, lse = H.token_logprobs(x, y, temperature=0.75)
    R.assert_near(logp, want.logp, near, "logp")
    R.assert_near(lse, want.lse, R.LOGP + want.lse.abs().nan_to_num(0, 0, 0) * R.EPS, "lse")
    gen = torch.Generator().manual_seed(4)
    old = (want.logp.nan_to_num(0.0, 0.0, -3.0) + 0.05).float()
    adv, w = torch.randn(rows, generator=gen), torch.rand(rows, generator=gen)
    total, loss, kl, g = R.policy(want, old, adv, w, None, 0.2, 0.2, 0.0, 256.0)
    slope = (torch.exp(want.logp - old.double()).nan_to_num(0, 0, 0) * adv.double()).abs()
    delta = slope * R.LOGP * w.double() * 256.0 + g.abs().nan_to_num(0, 0, 0) * 4 * R.EPS
    tol = grad_tolerance(want, g, dtype, delta).nan_to_num(0, 0, 0)
    args = (old.to(dev()), adv.to(dev()), w.to(dev()))
    plain = H.policy_loss(x, y, *args, temperature=0.75, with_grad=False)
    got = H.policy_loss(x, y, *args, temperature=0.75, grad_scale=256.0)
    R.assert_near(got.token_loss, loss, slope * R.LOGP + loss.abs().nan_to_num(0, 0, 0) * R.EPS, "token_loss")
    R.assert_near(got.grad, want.grad(g), tol, "grad")
    assert torch.equal(plain.token_loss.nan_to_num(), got.token_loss.nan_to_num()) and plain.grad is None
    y[8] = y[9] = y[13] = y[15] = -1  # the NaN rows
    cu = torch.tensor([0, 3, 10, 16, 20])
    want = R.Rows(x, y, 0.75)
    ref = want.logp.nan_to_num(0.0, 0.0, -3.0).float() - 0.1
    keep = torch.isfinite(want.logp)
    y[~keep.to(dev())] = -1
    want = R.Rows(x, y, 0.75)
    loss, losses, rewards, g = R.preference(want, cu, ref, 0.2, 0.0, 256.0)
    out = H.preference_loss(x, y, cu.to(dev()), ref.to(dev()), beta=0.2, temperature=0.75, grad_scale=256.0, grad_out=x)
    d_reward = 0.2 * (cu[1:] - cu[:-1]).double() * R.LOGP
    R.assert_near(out.rewards, rewards, d_reward + rewards.abs() * R.EPS, "rewards")
    delta = torch.full((rows,), 256.0 * 0.2 / 2 * float(d_reward.max()) / 2, dtype=torch.float64) + g.abs() * 4 * R.EPS
    R.assert_near(out.grad, want.grad(g), grad_tolerance(want, g, dtype, delta), "pair grad")
