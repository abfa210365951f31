"""Cases of the training operators: log-probabilities, preference and policy losses, gradient clipping.

Where ``own`` is false, ``run`` computes each operator in elementary torch
operations; where it is true, it calls the framework.
"""

import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
CLIP_LOW, CLIP_HIGH, KL, BETA, SMOOTHING = 0.2, 0.25, 0.05, 0.1, 0.05


def listed():
    return [
        # one decision scored while serving: latency alone counts
        {"name": "logprobs_one_row", "op": "logprobs", "dtype": "bf16", "rows": 1, "vocab": 1 << 15, "ignored": 0.0,
         "masked": False, "pad": 0, "temperature": 1.0, "backward": False},
        # scoring a batch of sessions with a frozen reference: a candidate count that no vector divides, rows inside wider ones
        {"name": "logprobs_odd_fp32", "op": "logprobs", "dtype": "fp32", "rows": 2047, "vocab": 50021, "ignored": 0.25,
         "masked": True, "pad": 3, "temperature": 0.75, "backward": False},
        # the gradient of the log-probabilities for a loss that the program computes itself
        {"name": "logprobs_backward", "op": "logprobs", "dtype": "bf16", "rows": 8192, "vocab": 1 << 16, "ignored": 0.25,
         "masked": False, "pad": 0, "temperature": 1.0, "backward": True},
        # a few pairs of short sessions over a short candidate list, as online training in small steps has them
        {"name": "preference_small", "op": "preference", "dtype": "fp32", "pairs": 4, "length": 24, "vocab": 1 << 12,
         "ignored": 0.3, "masked": True, "pad": 0, "temperature": 1.0},
        # an ordinary step
        {"name": "preference_ordinary", "op": "preference", "dtype": "bf16", "pairs": 16, "length": 256, "vocab": 1 << 15,
         "ignored": 0.4, "masked": False, "pad": 0, "temperature": 1.0},
        # half precision under a loss scale, an odd candidate count, ragged sessions
        {"name": "preference_odd_fp16", "op": "preference", "dtype": "fp16", "pairs": 37, "length": 61, "vocab": 40009,
         "ignored": 0.2, "masked": False, "pad": 0, "temperature": 0.875},
        # the largest step: offsets past 32 bits
        {"name": "preference_large", "op": "preference", "dtype": "bf16", "pairs": 16, "length": 512, "vocab": 1 << 17,
         "ignored": 0.25, "masked": False, "pad": 0, "temperature": 1.0},
        # slates of a thousand sampled candidates
        {"name": "policy_slates_fp32", "op": "policy", "dtype": "fp32", "seqs": 16, "length": 32, "vocab": 1000,
         "ignored": 0.0, "masked": True, "pad": 0, "temperature": 1.0, "kl": True},
        # an ordinary step with prompts left out, rows that no vector divides
        {"name": "policy_odd_bf16", "op": "policy", "dtype": "bf16", "seqs": 24, "length": 171, "vocab": 50021,
         "ignored": 0.4, "masked": False, "pad": 0, "temperature": 0.75, "kl": True},
        # the largest step, without a reference
        {"name": "policy_large_fp16", "op": "policy", "dtype": "fp16", "seqs": 32, "length": 384, "vocab": 1 << 17,
         "ignored": 0.1, "masked": False, "pad": 0, "temperature": 1.0, "kl": False},
        # the gradients of a small step, which the bound does not touch
        {"name": "clip_small", "op": "clip", "small": 6, "dense": 2, "width": 256, "rows": 4096, "dim": 64, "dtype": "fp32",
         "clipped": False},
        # dense weights in bf16 beside 2^20 found rows of 64 floats, clipped into the optimiser's own buffers
        {"name": "clip_large", "op": "clip", "small": 256, "dense": 60, "width": 2048, "rows": 1 << 20, "dim": 64,
         "dtype": "bf16", "clipped": True},
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["logprobs", "preference", "policy", "clip"])
    if op == "clip":
        return {"op": op, "small": rng.randint(1, 200), "dense": rng.randint(0, 40), "width": _spread(rng, 16, 2047),
                "rows": _spread(rng, 1, 1 << 20), "dim": rng.choice([1, 8, 16, 32, 64, 65, 128]),
                "dtype": rng.choice(["fp32", "bf16", "fp16"]), "clipped": rng.random() < 0.7}
    case = {"op": op, "dtype": rng.choice(["fp32", "bf16", "bf16", "fp16"]), "vocab": _spread(rng, 8, 1 << 18),
            "ignored": round(rng.uniform(0.0, 0.6), 2), "masked": rng.random() < 0.3, "pad": rng.choice([0, 0, 1, 8, 64]),
            "temperature": rng.choice([1.0, 1.0, 0.5, 0.75, 1.25])}
    most = min(1 << 15, (1 << 29) // case["vocab"])
    tokens = _spread(rng, 1, max(1, most))
    if op == "logprobs":
        return {**case, "rows": tokens, "backward": rng.random() < 0.5}
    length = _spread(rng, 1, max(1, min(tokens // 2, 2000)))
    many = max(1, tokens // length)
    if op == "preference":
        return {**case, "pairs": max(1, many // 2), "length": length}
    return {**case, "seqs": many, "length": length, "kl": rng.random() < 0.5}


def _lengths(case):
    """The ragged lengths of a case's sequences: between half the mean and one and a half."""
    many = 2 * case["pairs"] if case["op"] == "preference" else case["seqs"]
    mean = case["length"]
    r = random.Random(many * 1000003 + mean)
    return [r.randint((mean + 1) // 2, mean + mean // 2) for _ in range(many)]


def _prompt(case, n):
    """How many leading tokens of a sequence of n have no label."""
    return int(case["ignored"] * n)


def _sequences(case):
    return [case["rows"]] if case["op"] == "logprobs" else _lengths(case)


def _scale(case):
    """fp16 gradients are held under a loss scale, which undoes the mean over rows, pairs or sequences."""
    if case["dtype"] != "fp16":
        return 1.0
    many = {"logprobs": "rows", "preference": "pairs", "policy": "seqs"}[case["op"]]
    return 2.0 ** int(math.log2(256 * case[many]))


def _logits(case, gen, dev):
    lengths = _sequences(case)
    rows, vocab = sum(lengths), case["vocab"]
    x = torch.randn(rows, vocab + case["pad"], dtype=DTYPES[case["dtype"]], device=dev, generator=gen)
    x = x.mul_(2.5)[:, :vocab]
    live = torch.full((rows,), vocab, dtype=torch.int64, device=dev)
    if case["masked"]:  # candidate lists of unequal length: what is past a row's end is -inf
        live = torch.randint(vocab // 4 + 1, vocab + 1, (rows,), device=dev, generator=gen)
    labels = (torch.rand(rows, device=dev, generator=gen, dtype=torch.float64) * live).to(torch.int64).clamp_(max=vocab - 1)
    at = torch.arange(rows, device=dev)
    x[at, labels] += (0.5 * math.log(vocab) + 1.5 * torch.randn(rows, device=dev, generator=gen)).to(x.dtype)  # a trained model's
    if case["masked"]:
        if rows >= 64:
            live[63::64] = 0  # rows with no candidate at all
        x.masked_fill_(torch.arange(vocab, device=dev) >= live[:, None], -math.inf)
    told = torch.tensor([t >= _prompt(case, n) for n in lengths for t in range(n)], dtype=torch.bool, device=dev)
    labels[~told] = -100
    return x, labels, lengths


def _kept_logp(x, labels, temperature):
    """Log-probabilities and their normalisers as an earlier call of the program left them."""
    lse = torch.logsumexp(x.float() / temperature, 1)
    logp = x.gather(1, labels.clamp(min=0)[:, None])[:, 0].float() / temperature - lse
    out = (labels < 0) | torch.isinf(lse)
    return logp.masked_fill_(out, 0.0), lse.masked_fill_(labels < 0, 0.0)


def _sizes(case):
    """Elements of each gradient: biases and norms of any length, dense weights, the found rows (always fp32)."""
    r = random.Random(case["small"] * 7 + case["dense"] * 1009 + case["width"])
    w = case["width"]
    towers = [r.randint(1, 4 * w) for _ in range(case["small"])] + [w * r.randint(w, 4 * w) for _ in range(case["dense"])]
    return towers, [case["rows"] * case["dim"]]


def _gradients(case, gen, dev):
    """Gradients as views of flat buffers, and buffers like them for the clipped ones."""
    towers, rows = _sizes(case)
    flats = [torch.randn(sum(towers), dtype=DTYPES[case["dtype"]], device=dev, generator=gen).mul_(1e-2),
             torch.randn(sum(rows), device=dev, generator=gen).mul_(1e-2)]
    outs = [torch.zeros_like(f) for f in flats]
    views, copies = ([v for f, n in zip(fs, (towers, rows)) for v in f.split(n)] for fs in (flats, outs))
    norm = 1e-2 * math.sqrt(sum(towers) + sum(rows))
    return {"grads": views, "flats": flats, "outs": outs, "copies": copies, "max_norm": norm * (0.3 if case["clipped"] else 3.0)}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if case["op"] == "clip":
        return {"case": case, **_gradients(case, gen, dev)}
    x, labels, lengths = _logits(case, gen, dev)
    rows, tau = x.shape[0], case["temperature"]
    s = {"case": case, "x": x, "labels": labels}
    if case["op"] == "logprobs":
        if case["backward"]:
            s["lse"] = _kept_logp(x, labels, tau)[1]
            s["g"] = torch.randn(rows, device=dev, generator=gen).mul_(_scale(case) / rows)
        return s
    logp = _kept_logp(x, labels, tau)[0]
    if case["op"] == "preference":
        s["cu"] = torch.tensor([0] + [sum(lengths[:i + 1]) for i in range(len(lengths))], dtype=torch.int64, device=dev)
        # the policy has moved from the reference, up for chosen and down for rejected sessions, by a few units in all
        moved = [(2.0 if i % 2 == 0 else -3.0) / n for i, n in enumerate(lengths) for _ in range(n)]
        noise = torch.randn(rows, device=dev, generator=gen).mul_(0.7 / math.sqrt(case["length"]))
        s["ref"] = logp - torch.tensor(moved, dtype=torch.float32, device=dev) + noise
        return s
    # the old policy is a few updates back: some ratios pass the bounds, none lies on one
    d = 0.15 * torch.randn(rows, device=dev, generator=gen)
    for border in (math.log(1.0 - CLIP_LOW), math.log(1.0 + CLIP_HIGH)):
        d = torch.where((d - border).abs() < 1e-3, d + 2e-3, d)
    s["old"] = logp - d
    s["ref"] = logp + 0.1 * torch.randn(rows, device=dev, generator=gen) if case["kl"] else None
    s["adv"] = torch.randn(rows, device=dev, generator=gen)
    told = [n - _prompt(case, n) for n in lengths]
    w = [1.0 / (max(1, k) * len(lengths)) for n, k in zip(lengths, told) for _ in range(n)]
    s["w"] = torch.tensor(w, dtype=torch.float32, device=dev).masked_fill_(labels < 0, 0.0)
    return s


# The plain forms.


def _rows(x, labels, tau):
    """Row-wise softmax: label positions, rows that count, normalisers, log-probabilities, probabilities and 1 less the
    label's. Elements are in 32 bits, taken from each row's maximum; their long sum, and the few values a row whose
    differences count, in 64."""
    at = labels.clamp(min=0)
    label = x.gather(1, at[:, None])[:, 0].double() / tau
    x = x.float()
    top = x.amax(1)
    counts = (labels >= 0) & (top != -math.inf)
    top = torch.where(counts, top, torch.zeros_like(top))
    e = ((x - top[:, None]) / tau).exp()
    total = e.sum(1, dtype=torch.float64)
    rest = 1.0 - e.gather(1, at[:, None])[:, 0].double() / total
    lse = top.double() / tau + total.log()
    return at, counts, lse, torch.where(counts, label - lse, torch.zeros_like(lse)), e / total.float()[:, None], rest


def _dlogits(p, rest, at, counts, g, kind):
    """g (1[label] - p), zero in the rows that do not count."""
    d = -g[:, None] * p
    d.scatter_(1, at[:, None], (g * rest).float()[:, None])
    return torch.where(counts[:, None], d, torch.zeros_like(d)).to(kind)


def _plain_logprobs(s):
    x, tau, labels = s["x"], s["case"]["temperature"], s["labels"]
    if s["case"]["backward"]:
        at = labels.clamp(min=0)
        p = (x.float() / tau - s["lse"][:, None]).exp()
        rest = -torch.expm1(x.gather(1, at[:, None])[:, 0].double() / tau - s["lse"])
        return _dlogits(p, rest, at, (labels >= 0) & (s["lse"] != -math.inf), s["g"] / tau, x.dtype)
    _, _, lse, logp, _, _ = _rows(x, labels, tau)
    return [logp.float(), torch.where(labels >= 0, lse, torch.zeros_like(lse)).float()]


def _softplus(m):
    return m.clamp(min=0) + (1.0 + (-m.abs()).exp()).log()


def _plain_preference(s):
    tau, cu = s["case"]["temperature"], s["cu"]
    at, counts, _, logp, p, rest = _rows(s["x"], s["labels"], tau)
    ratio = torch.where(counts, logp - s["ref"], torch.zeros_like(logp))
    run_to = torch.cat([ratio.new_zeros(1), ratio.cumsum(0)])
    rewards = BETA * (run_to[cu[1:]] - run_to[cu[:-1]])
    m = rewards[0::2] - rewards[1::2]
    losses = (1.0 - SMOOTHING) * _softplus(-m) + SMOOTHING * _softplus(m)
    c = BETA / m.numel() * (1.0 / (1.0 + (-m).exp()) - 1.0 + SMOOTHING)
    c = torch.stack([c, -c], 1).reshape(-1)
    g = (_scale(s["case"]) / tau * c).repeat_interleave(cu[1:] - cu[:-1], output_size=logp.numel()).float()
    grad = _dlogits(p, rest, at, counts, g, s["x"].dtype)
    return [losses.mean().float(), losses.float(), rewards.float(), logp.float(), grad]


def _plain_policy(s):
    tau = s["case"]["temperature"]
    at, counts, _, logp, p, rest = _rows(s["x"], s["labels"], tau)
    zero = torch.zeros_like(logp)
    r = (logp - s["old"]).exp()
    free, bound = r * s["adv"], r.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * s["adv"]
    loss = -torch.minimum(free, bound)
    g = torch.where(free <= bound, -free, zero)
    kl = zero
    if s["ref"] is not None:
        d = s["ref"] - logp
        kl = torch.where(counts, torch.expm1(d) - d, zero)
        loss = loss + KL * kl
        g = g - KL * torch.expm1(d)
    loss = torch.where(counts, loss, zero)
    g = (s["w"] * g * (_scale(s["case"]) / tau)).float()
    grad = _dlogits(p, rest, at, counts, g, s["x"].dtype)
    return [(s["w"] * loss).sum().float(), loss.float(), kl.float(), logp.float(), grad]


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    c = (s["max_norm"] / norm).clamp(max=1.0)
    to = s["copies"] if s["case"]["clipped"] else s["grads"]
    _ = [o.copy_(g.float() * c) for o, g in zip(to, s["grads"])]
    return [norm] + (s["outs"] if s["case"]["clipped"] else s["flats"])


def _own(s):
    """The framework's calls."""
    import hash_table_cache_amd as H

    case = s["case"]
    if case["op"] == "clip":
        norm = H.clip_grad_norm(s["grads"], s["max_norm"], out=s["copies"] if case["clipped"] else None)
        return [norm] + (s["outs"] if case["clipped"] else s["flats"])
    tau = case["temperature"]
    if case["op"] == "logprobs":
        if case["backward"]:
            return H.token_logprobs_backward(s["x"], s["labels"], s["lse"], s["g"], temperature=tau)
        return list(H.token_logprobs(s["x"], s["labels"], temperature=tau))
    if case["op"] == "preference":
        return list(H.preference_loss(s["x"], s["labels"], s["cu"], s["ref"], beta=BETA, label_smoothing=SMOOTHING,
                                      temperature=tau, grad_scale=_scale(case)))
    return list(H.policy_loss(s["x"], s["labels"], s["old"], s["adv"], s["w"], s["ref"], clip_low=CLIP_LOW,
                              clip_high=CLIP_HIGH, kl_coef=KL if case["kl"] else 0.0, temperature=tau,
                              grad_scale=_scale(case)))


def run(state):
    if own:
        return _own(state)
    return {"logprobs": _plain_logprobs, "preference": _plain_preference, "policy": _plain_policy,
            "clip": _plain_clip}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "clip":
        towers, rows = (sum(n) for n in _sizes(case))
        size, n = SIZE[case["dtype"]] * towers + 4 * rows, towers + rows
        # gradients that the bound leaves as they are need no writing
        return {"bytes": size * (2 if case["clipped"] else 1), "flops": (3 if case["clipped"] else 2) * n}
    lengths = _sequences(case)
    rows, told = sum(lengths), sum(n - _prompt(case, n) for n in lengths)
    row = case["vocab"] * SIZE[case["dtype"]]
    back = case["op"] != "logprobs" or case["backward"]
    read, written = told * row, rows * row if back else 0
    per_row = {"logprobs": 20, "preference": 16, "policy": 32}[case["op"]]
    return {"bytes": read + written + rows * per_row, "flops": told * case["vocab"] * (8 if back else 4)}


# The definition in 64 bits.


def _exact_rows(x, labels, tau, per_row):
    """per_row(first, last, scaled logits, label, row counts) over blocks of rows; its results joined."""
    many = max(1, (1 << 25) // x.shape[1])

    def block(a):
        z, y = x[a:a + many].double() / tau, labels[a:a + many]
        return per_row(a, min(a + many, x.shape[0]), z, y.clamp(min=0), (y >= 0) & ~(z == -math.inf).all(1))

    return torch.cat([block(a) for a in range(0, x.shape[0], many)])


def _exact_logp(x, labels, tau):
    def take(a, b, z, y, ok):
        return torch.log_softmax(z, 1).gather(1, y[:, None])[:, 0].masked_fill(~ok, 0.0)

    return _exact_rows(x, labels, tau, take)


def _exact_grad(x, labels, tau, g, lse=None):
    def take(a, b, z, y, ok):
        d = torch.softmax(z, 1).neg_() if lse is None else torch.exp(z - lse[a:b].double()[:, None]).neg_()
        d[torch.arange(b - a, device=d.device), y] += 1.0
        return d.mul_((g[a:b] / tau)[:, None]).masked_fill_(~ok[:, None], 0.0)

    return _exact_rows(x, labels, tau, take)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(f.double().square().sum()) for f in s["flats"]))
        c = min(1.0, s["max_norm"] / norm)
        return [torch.tensor(norm, dtype=torch.float64)] + [f.double() * c for f in s["flats"]]
    x, y, tau = s["x"], s["labels"], case["temperature"]
    if case["op"] == "logprobs":
        if case["backward"]:
            return _exact_grad(x, y, tau, s["g"].double(), s["lse"])
        lse = _exact_rows(x, y, tau, lambda a, b, z, at, ok: torch.logsumexp(z, 1).masked_fill(y[a:b] < 0, 0.0))
        return [_exact_logp(x, y, tau), lse]
    logp = _exact_logp(x, y, tau)
    ok = (y >= 0) & (x != -math.inf).any(1)
    if case["op"] == "preference":
        lengths = _lengths(case)
        seq = torch.arange(len(lengths), device=x.device).repeat_interleave(torch.tensor(lengths, device=x.device))
        ratio = (logp - s["ref"].double()).masked_fill(~ok, 0.0)
        rewards = BETA * torch.zeros(len(lengths), dtype=torch.float64, device=x.device).index_add_(0, seq, ratio)
        m = rewards.view(-1, 2)[:, 0] - rewards.view(-1, 2)[:, 1]
        logsig = torch.nn.functional.logsigmoid
        losses = -(1 - SMOOTHING) * logsig(m) - SMOOTHING * logsig(-m)
        slope = -(1 - SMOOTHING) * torch.sigmoid(-m) + SMOOTHING * torch.sigmoid(m)
        sign = 1.0 - 2.0 * (seq % 2).double()
        g = _scale(case) * BETA / len(m) * slope[seq // 2] * sign
        return [losses.mean(), losses, rewards, logp, _exact_grad(x, y, tau, g)]
    l = logp.detach().requires_grad_()
    with torch.enable_grad():
        r = torch.exp(l - s["old"].double())
        a = s["adv"].double()
        loss = -torch.where(a >= 0, torch.clamp(r, max=1 + CLIP_HIGH), torch.clamp(r, min=1 - CLIP_LOW)) * a
        kl = torch.zeros_like(loss)
        if s["ref"] is not None:
            d = s["ref"].double() - l
            kl = torch.exp(d) - 1 - d
            loss = loss + KL * kl
        loss, kl = loss.masked_fill(~ok, 0.0), kl.masked_fill(~ok, 0.0)
        total = (s["w"].double() * loss).sum()
        g = torch.autograd.grad(total, l)[0]
    return [total.detach(), loss.detach(), kl.detach(), logp, _exact_grad(x, y, tau, g * _scale(case))]
