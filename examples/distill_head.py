"""From logits to updated parameters: a student head distilled from a teacher, its parameters stepped as shards.

Each of N virtual ranks has its own rows of hidden states. Per step and rank: the teacher's top log probabilities
(ss_token_logprobs), the student's logits, the loss and its gradient in one call (ss_distill_topk, the gradient written
over the logits), and the head's 16-bit gradient. The ranks' gradients then go through the shard step: the clip norm over
all shards, the fused reduce + AdamW + cast of every shard, and the unshard into the flat unit that the next step reads.

    python examples/distill_head.py [--steps 30] [--vocab 50257] [--dim 256] [--rows 512] [--ranks 4] [--top 32]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fsdp_sharded_mixed_ss_gb300 as ss  # noqa: E402


class Head:
    """A vocabulary head (vocab, dim) as one flat 16-bit unit cut into shards, with fp32 state per shard."""

    def __init__(self, vocab: int, dim: int, n_ranks: int, device, seed: int):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.vocab, self.dim = vocab, dim
        _, self.bounds = ss.ss_flatten_layout([vocab * dim], n_ranks)
        w = torch.randn(vocab * dim, generator=g, device=device) * 0.02
        self.flat = w.to(torch.bfloat16)
        cuts = [(int(a), int(b)) for a, b in zip(self.bounds[:-1], self.bounds[1:])]
        self.cuts = cuts
        self.master = [w[a:b].clone() for a, b in cuts]
        self.m = [torch.zeros(b - a, device=device) for a, b in cuts]
        self.v = [torch.zeros(b - a, device=device) for a, b in cuts]
        self.shards = [torch.empty(b - a, dtype=torch.bfloat16, device=device) for a, b in cuts]
        self.sumsq = torch.zeros(n_ranks, dtype=torch.float64, device=device)
        self.coef = torch.zeros(1, device=device)
        self.work = torch.empty(max(ss.ss_grad_sumsq_workspace(b - a) for a, b in cuts) // 8, dtype=torch.float64,
                                device=device)

    @property
    def weight(self):
        return self.flat.view(self.vocab, self.dim)

    def step(self, rank_grads, t: int, lr: float, max_norm: float) -> None:
        """One update from the ranks' flat 16-bit gradients, summed with equal weights."""
        scale = 1.0 / len(rank_grads)
        for k, (a, b) in enumerate(self.cuts):
            ss.ss_grad_sumsq(b - a, self.sumsq[k:], self.work, rank_grads=[g[a:b] for g in rank_grads],
                             post_scale=scale)
        ss.ss_clip_coef(self.sumsq, len(self.cuts), max_norm, self.coef)
        hp = dict(lr=lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=t)
        for k, (a, b) in enumerate(self.cuts):
            ss.ss_adam_step(hp, b - a, self.master[k], self.m[k], self.v[k], rank_grads=[g[a:b] for g in rank_grads],
                            post_scale=scale, param16=self.shards[k], dev_grad_scale=self.coef)
        ss.ss_unshard(self.shards, self.bounds, self.flat)


def train(steps=30, vocab=50257, dim=256, rows=512, n_ranks=4, top=32, lr=2e-3, device="cuda"):
    """(mean loss of every step, mean log probability of the teacher's choices before, and after)."""
    g = torch.Generator(device=device)
    g.manual_seed(7)
    student = Head(vocab, dim, n_ranks, device, seed=1)
    teacher = (torch.randn((vocab, dim), generator=g, device=device) * 0.25).to(torch.bfloat16)
    hidden = [torch.randn((rows, dim), generator=g, device=device).to(torch.bfloat16) for _ in range(n_ranks)]
    f32 = dict(dtype=torch.float32, device=device)
    lists = []
    for h in hidden:  # the teacher's pass: its top log probabilities are the students' lists
        ids = torch.empty((rows, top), dtype=torch.int32, device=device)
        lps = torch.empty((rows, top), **f32)
        ss.ss_token_logprobs(h @ teacher.t(), top_logprob=lps, top_id=ids)
        lists.append((ids, lps))

    def choices():
        lp = torch.empty(rows, **f32)
        total = 0.0
        for h, (ids, _) in zip(hidden, lists):
            ss.ss_token_logprobs(h @ student.weight.t(), ids[:, 0].contiguous(), logprob=lp)
            total += float(lp.mean())
        return total / n_ranks

    before = choices()
    weight = torch.full((rows,), 1.0 / rows, **f32)
    loss = torch.empty((n_ranks, rows), **f32)
    means = []
    for t in range(1, steps + 1):
        grads = []
        for r, (h, (ids, lps)) in enumerate(zip(hidden, lists)):
            z = h @ student.weight.t()
            ss.ss_distill_topk(z, ids, lps, loss[r], d_logits=z, row_weight=weight, tail=ss.SS_TAIL_BUCKET)
            grads.append((z.t() @ h).reshape(-1))
        student.step(grads, t, lr, max_norm=10.0)
        means.append(float(loss.sum()) / n_ranks)
    return means, before, choices()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--vocab", type=int, default=50257)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--top", type=int, default=32)
    a = ap.parse_args()
    means, before, after = train(a.steps, a.vocab, a.dim, a.rows, a.ranks, a.top)
    print(f"divergence {means[0]:.4f} -> {means[-1]:.4f} over {a.steps} steps; "
          f"mean log probability of the teacher's choices {before:.3f} -> {after:.3f}")


if __name__ == "__main__":
    main()
