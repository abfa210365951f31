"""Online training of stored embeddings from feedback.

Item embeddings live in a table. Every step finds the rows of a candidate list
(inserting new items), scores sessions against them, turns feedback into
gradients, bounds them, and assigns the rows back:

    find_or_insert -> logits -> preference_loss / policy_loss -> clip_grad_norm -> assign

Two kinds of feedback take turns: pairs of sessions of which one was preferred
(against a frozen copy of the model), and sessions with a reward (against the
model that served them). Synthetic users prefer the items of one half. With
--entropy, steps on rewards also hold up the entropy of the scores
(token_stats and its gradient), which is printed beside the three items scored
highest; with --muon, the dense weight moves by an orthogonalised momentum step
(muon_update) in place of a scaled gradient.

    python examples/online_feedback.py [--steps 40] [--items 2000] [--dim 64] [--entropy 0.01] [--muon 0.02]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import hash_table_cache_amd as H  # noqa: E402


def sessions(count, length, items, liked, gen, dev):
    """Labels of `count` sessions, a row each: items that users like (even
    numbers) or not (odd ones)."""
    picks = torch.randint(0, items // 2, (count, length), generator=gen, device=dev)
    return (2 * picks + (0 if liked else 1)).reshape(-1)


def train(steps=40, items=2000, dim=64, pairs=16, length=12, lr=8.0, seed=0, verbose=False, entropy=0.0, muon=0.0):
    """Returns the losses of the two kinds of step, in order. entropy: what a nat
    of it is worth, averaged over tokens; muon: the rate of the orthogonalised steps."""
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(seed)
    table = H.HashTable(capacity=1 << 14, dim=dim)
    keys = torch.arange(1, items + 1, dtype=torch.int64, device=dev)
    context = torch.randn(2 * pairs * length, dim, generator=gen, device=dev)  # what the sessions' model sees
    weight = torch.eye(dim, device=dev)  # its dense part
    fresh = 0.1 * torch.randn(items, dim, generator=gen, device=dev)
    rows, _ = table.find_or_insert(keys, fresh.clone(), torch.zeros_like(keys))
    frozen, frozen_weight = rows.clone(), weight.clone()
    cu = torch.arange(2 * pairs + 1, dtype=torch.int64, device=dev) * length
    tokens = 2 * pairs * length
    preference, policy = [], []
    momentum = torch.zeros_like(weight)
    stats = None
    for step in range(steps):
        rows, found, _ = table.find(keys)
        hidden = context @ weight
        logits = (hidden @ rows.t()).to(torch.bfloat16)
        spread = None
        if step % 2 == 0:
            good = sessions(pairs, length, items, True, gen, dev).view(pairs, length)
            bad = sessions(pairs, length, items, False, gen, dev).view(pairs, length)
            labels = torch.stack([good, bad], 1).reshape(-1)  # sessions 2p and 2p + 1
            reference = ((context @ frozen_weight) @ frozen.t()).to(torch.bfloat16)
            ref_logp, _ = H.token_logprobs(reference, labels)
            out = H.preference_loss(logits, labels, cu, ref_logp, beta=0.2, grad_out=logits)
            preference.append(out.loss)
        else:
            labels = sessions(2 * pairs, length, items, True, gen, dev)
            odd = torch.rand(tokens, generator=gen, device=dev) < 0.5
            labels = torch.where(odd, labels + 1, labels)
            reward = torch.where(odd, -1.0, 1.0)
            if entropy:
                stats = H.token_stats(logits, labels, 3)
                served = stats.logp
                each = torch.full((tokens,), -entropy / tokens, device=dev)  # the loss falls with it
                spread = H.token_stats_backward(logits, labels, stats.lse, stats.entropy, grad_entropy=each)
            else:
                served, _ = H.token_logprobs(logits, labels)  # the policy that served is the present one
            out = H.policy_loss(logits, labels, served, reward, torch.full((tokens,), 1.0 / tokens, device=dev), served,
                                kl_coef=0.05, grad_out=logits)
            policy.append(out.loss)
        dlogits = out.grad.float()  # in the logits' place
        if spread is not None:
            dlogits += spread.float()
        drows, dhidden = dlogits.t() @ hidden, dlogits @ rows
        dweight = context.t() @ dhidden
        H.clip_grad_norm([drows, dweight], 1.0)
        if muon:
            H.muon_update([weight], [dweight], [momentum], muon, momentum=0.9)
        else:
            weight -= 0.02 * lr * dweight
        table.assign(keys, rows - lr * drows, torch.full_like(keys, step + 1))
    result = [float(v) for v in preference], [float(v) for v in policy]
    table.close()
    if verbose:
        for name, losses in zip(("preference loss", "policy loss"), result):
            print(name, " ".join(f"{v:.4f}" for v in losses))
        if stats is not None:
            print(f"entropy {float(stats.entropy.mean()):.4f}, first session's items and their log-probabilities",
                  list(zip(stats.top_ids[0].tolist(), (round(v, 3) for v in stats.top_logp[0].tolist()))))
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--items", type=int, default=2000)
    ap.add_argument("--dim", type=int, default=64)
    ap.add_argument("--entropy", type=float, default=0.0)
    ap.add_argument("--muon", type=float, default=0.0)
    a = ap.parse_args()
    train(a.steps, a.items, a.dim, verbose=True, entropy=a.entropy, muon=a.muon)
