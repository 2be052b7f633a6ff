"""A tied embedding and head trained by a clipped policy loss, its table stepped as shards.

A bigram policy: the next token's logits are h W^T with h = s W[previous token], one table W for both ends. Every round,
each of N virtual ranks samples tokens for its own rows (ss_embedding, the logits, ss_token_logprobs) and takes a few
updates on them. Per update and rank: the lookup out of the flat unit, the logits, the loss with a KL term against the
table of the start and its gradient over the logits (ss_policy_loss), and the table's gradient: the head's part by a
product, the embedding's on top of it, summed over the rows of each token (ss_embedding_grad, in place). The ranks'
gradients then go through the shard step of examples/distill_head.py.

    python examples/tied_policy.py [--rounds 20] [--updates 4] [--vocab 257] [--dim 64] [--rows 512] [--ranks 4]
"""
from __future__ import annotations

import argparse
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [HERE, os.path.dirname(HERE)]

import torch  # noqa: E402

import fsdp_sharded_mixed_ss_gb300 as ss  # noqa: E402
from distill_head import Head  # noqa: E402


def hidden_of(table, tokens, scale):
    h = torch.empty((tokens.numel(), table.shape[1]), dtype=table.dtype, device=table.device)
    ss.ss_embedding(table, tokens, h, scale=scale)
    return h


def table_gradient(table, previous, batch, scale, workspace, *, kl_coef=0.02, entropy_coef=0.001):
    """(losses of the rows, gradient of their sum with respect to the table, flat, of the table's type) of one rank."""
    h = hidden_of(table, previous, scale)
    z = h @ table.t()
    loss = torch.empty(previous.numel(), device=table.device)
    ss.ss_policy_loss(z, batch["tokens"], batch["advantage"], loss, old_logprob=batch["old"],
                      ref_logprob=batch["reference"], row_weight=batch["weight"], kl_coef=kl_coef,
                      entropy_coef=entropy_coef, d_logits=z)
    d_h = z @ table
    d_table = z.t() @ h
    ss.ss_embedding_grad(d_h, previous, d_table, workspace, base=d_table, scale=scale)
    return loss, d_table.reshape(-1)


def log_probs(table, previous, tokens, scale):
    lp = torch.empty(tokens.numel(), device=table.device)
    ss.ss_token_logprobs(hidden_of(table, previous, scale) @ table.t(), tokens, logprob=lp)
    return lp


def train(rounds=20, updates=4, vocab=257, dim=64, rows=512, n_ranks=4, lr=5e-3, device="cuda"):
    """Mean reward of every round's samples: 1 for an even token behind an even one or an odd one behind an odd one."""
    g = torch.Generator(device=device)
    g.manual_seed(11)
    scale = 12.0
    policy = Head(vocab, dim, n_ranks, device, seed=3)
    start = policy.weight.clone()
    workspace = torch.empty(ss.ss_embedding_grad_workspace(rows, vocab, dim), dtype=torch.uint8, device=device)
    weight = torch.full((rows,), 1.0 / rows, device=device)
    rewards, t = [], 0
    for _ in range(rounds):
        batches = []
        for _ in range(n_ranks):
            previous = torch.randint(0, vocab, (rows,), generator=g, device=device)
            p = torch.softmax((hidden_of(policy.weight, previous, scale) @ policy.weight.t()).float(), dim=1)
            tokens = torch.multinomial(p, 1, generator=g)[:, 0]
            reward = ((tokens + previous + 1) % 2).float()
            batches.append((previous, dict(
                tokens=tokens, advantage=reward - reward.mean(), weight=weight, reward=reward,
                old=log_probs(policy.weight, previous, tokens, scale),
                reference=log_probs(start, previous, tokens, scale))))
        for _ in range(updates):
            t += 1
            policy.step([table_gradient(policy.weight, previous, b, scale, workspace)[1] for previous, b in batches],
                        t, lr, max_norm=1.0)
        rewards.append(sum(float(b["reward"].mean()) for _, b in batches) / n_ranks)
    return rewards


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=20)
    ap.add_argument("--updates", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=257)
    ap.add_argument("--dim", type=int, default=64)
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--ranks", type=int, default=4)
    a = ap.parse_args()
    rewards = train(a.rounds, a.updates, a.vocab, a.dim, a.rows, a.ranks)
    print("mean reward of a round's samples: " + " ".join(f"{r:.3f}" for r in rewards))


if __name__ == "__main__":
    main()
