"""The training operators together, as a step of learned rows uses them: rows
found in the table, logits, token statistics with alternatives, the gradient of
log-probability and entropy, clipping, the dense weight's momentum update, and
the rows assigned back; each against its formula in 64 bits on what it was given.
"""

import pathlib
import runpy

import pytest
import torch

import polar_reference as P
import training_reference as R
from conftest import gpu_available
from test_gpu_orthogonalize import update
from test_gpu_token_stats import backward_reference, check, dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_step(dtype):
    import hash_table_cache_amd as H

    items, dim, tokens, lr = 1500, 64, 96, 0.5
    gen = torch.Generator(device=dev()).manual_seed(4)
    table = H.HashTable(capacity=1 << 13, dim=dim)
    keys = torch.arange(1, items + 1, dtype=torch.int64, device=dev())
    table.insert_or_assign(keys, 0.3 * torch.randn(items, dim, generator=gen, device=dev()), torch.ones_like(keys))
    weight = torch.eye(dim, device=dev()) + 0.1 * torch.randn(dim, dim, generator=gen, device=dev())
    momentum = torch.zeros_like(weight)
    context = torch.randn(tokens, dim, generator=gen, device=dev())
    for step in range(3):
        rows, found, _ = table.find(keys)
        assert bool(found.all())
        hidden = context @ weight
        logits = (hidden @ rows.t()).to(dtype)
        labels = torch.randint(0, items, (tokens,), generator=gen, device=dev())
        labels[5] = -100
        logits[:, items // 2 + step:items // 2 + 200] = -torch.inf  # items that this step may not show
        labels = torch.where(labels >= items // 2, labels - items // 2, labels)
        st = check(logits, labels, 0.8, 10, f"step {step}")
        g = -torch.rand(tokens, generator=gen, device=dev()) / tokens
        ge = torch.full((tokens,), -0.01 / tokens, device=dev())
        ref, tol = backward_reference(logits, labels, 0.8, st.lse, st.entropy, g.cpu(), ge.cpu())
        ref[5] = 0.0
        dlogits = H.token_stats_backward(logits, labels, st.lse, st.entropy, g, ge, temperature=0.8, grad_out=logits)
        R.assert_near(dlogits, ref, tol, f"gradient {step}")
        d = dlogits.float()
        drows, dweight = d.t() @ hidden, context.t() @ (d @ rows)
        size = float(torch.sqrt(sum(R.f64(t).square().sum() for t in (drows, dweight))))
        before = R.f64(dweight)
        norm = H.clip_grad_norm([drows, dweight], 0.5 * size)
        assert abs(float(norm) - size) <= 8 * R.EPS * size
        # a factor and a product, each rounded once; the factor from a norm off by up to 8 steps
        R.assert_near(dweight, before * 0.5, before.abs() * 0.5 * 16 * R.EPS + R.TINY[torch.float32], f"clipped {step}")
        moved, want, tol = update(weight, dweight, momentum, 0.05, 1.0, 0.9, True, 0.01, 5, P.COEFFICIENTS, 1e-7)
        H.muon_update([weight], [dweight], [momentum], 0.05, momentum=0.9, weight_decay=0.01)
        R.assert_near(momentum, moved, moved.abs() * R.EPS + R.TINY[torch.float32], f"momentum {step}")
        P.assert_close(weight, want, tol, f"weight {step}")
        after = rows - lr * drows
        table.assign(keys, after, torch.full_like(keys, step + 2))
        assert torch.equal(table.find(keys)[0], after)
    table.close()


def test_a_captured_step():
    """Statistics, gradient, clipping and update in one graph, replayed on new logits beside eager work."""
    import hash_table_cache_amd as H

    tokens, vocab = 50, 9001
    gen = torch.Generator(device=dev()).manual_seed(5)
    logits = torch.randn(tokens, vocab, generator=gen, device=dev()).to(torch.bfloat16)
    labels = torch.randint(0, vocab, (tokens,), generator=gen, device=dev())
    g, ge = torch.randn(2, tokens, generator=gen, device=dev())
    state = [torch.randn(100, 140, generator=gen, device=dev()), torch.zeros(100, 140, device=dev())]
    grad = torch.randn(100, 140, generator=gen, device=dev())

    def step(logits, grad, state):
        st = H.token_stats(logits, labels, 4)
        d = H.token_stats_backward(logits, labels, st.lse, st.entropy, g, ge)
        norm = H.clip_grad_norm([d, grad], 1.0)
        H.muon_update([state[0]], [grad], [state[1]], 0.1)
        return [*st, d, norm]

    spare = [t.clone() for t in state]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(logits, grad.clone(), spare)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    held = [t.clone() for t in state]
    with torch.cuda.graph(graph):
        out = step(logits, grad, held)
    for h, t in zip(held, state):
        h.copy_(t)
    for k in range(4):
        logits.copy_(torch.randn(tokens, vocab, generator=gen, device=dev()) * (1 + k))
        grad.copy_(torch.randn(100, 140, generator=gen, device=dev()))
        own = grad.clone()
        graph.replay()
        want = step(logits, own, state)
        torch.cuda.synchronize()
        for p, q in zip((*out, grad, *held), (*want, own, *state)):
            assert torch.equal(p, q), k


def test_example_with_entropy_and_momentum():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "online_feedback.py"
    train = runpy.run_path(str(path))["train"]
    plain = train(steps=4, items=300, dim=32, pairs=4)
    again = train(steps=4, items=300, dim=32, pairs=4, entropy=0.0, muon=0.0)
    assert plain == again
    other = train(steps=4, items=300, dim=32, pairs=4, entropy=0.05, muon=0.01)
    values = [v for kind in other for v in kind]
    assert len(values) == 4 and all(v == v and abs(v) < 1e6 for v in values)
    assert other[0][0] == plain[0][0]  # the first step's loss is of the same scores
