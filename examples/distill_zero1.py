"""Distil a teacher's top logits into a small tied-embedding language model
trained with the ZeRO-1 step on N simulated ranks, end to end on one GPU.

The student is the two ends of a language model with nothing between them:
the rows of its embedding table are looked up, and the logits are their
products with the same (tied) table.  Each rank has its own tokens.  One step:

  lm_embedding         h = sqrt(D) * E[ids]            from the rank's weight slab
  torch.matmul         logits = h E^T / D
  lm_distill_step      loss and, in place of the logits, their gradient
  torch.matmul         the output layer's part of dE   into the rank's gradient slab
  lm_embedding_grad    the lookup's part of dE          added to it in place
  dp_zero1_step        reduce-scatter, clip, AdamW, all-gather

and at the end lm_logprobs scores tokens that the teacher likes best.

  python examples/distill_zero1.py [--steps 60] [--vocab 2000] [--width 128]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def train(steps=60, vocab=2000, width=128, tokens=512, ranks=4, top=16, temperature=2.0, seed=0,
          device="cuda"):
    """Returns the mean loss of each step, the replicas [ranks, vocab, width]
    and the mean log probability of the teacher's favourite tokens before and
    after."""
    import torch

    import gradient_reduction_zero_gb300.dpz as dpz

    V, D, T, N, K = vocab, width, tokens, ranks, top
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731

    # the arena: the table, padded to a multiple of 8 N elements
    P = -(-V * D // (8 * N)) * 8 * N
    weights = torch.zeros(N, P, dtype=torch.bfloat16, device=device)
    grads = torch.zeros(N, P, dtype=torch.bfloat16, device=device)
    master = torch.zeros(P, device=device)
    master[:V * D] = 0.02 * rand(V * D)
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    weights.copy_(master)                      # every replica the same
    norm, ws = torch.zeros(1, device=device), dpz.workspace(P, N, device)

    # the teacher: a fixed table of its own, of which the student sees the top K logits
    teacher = rand(V, 32)
    ids = torch.randint(0, V, (N, T), generator=g, device=device)
    t_logits, t_ids = torch.topk(teacher[ids] @ teacher.T, K, dim=2)

    scale = D ** 0.5
    h = torch.empty(T, D, dtype=torch.bfloat16, device=device)
    logits = torch.empty(T, V, dtype=torch.bfloat16, device=device)
    dh = torch.empty_like(h)
    loss, weight = torch.empty(T, device=device), torch.full((T,), 1.0 / T, device=device)
    emb_ws = dpz.lm_embedding_workspace(T, V, D, device)

    def forward(r):
        E = weights[r, :V * D].view(V, D)
        dpz.lm_embedding(E, ids[r], h, scale=scale)
        torch.matmul(h / D, E.T, out=logits)
        return E

    def score(r):
        """Mean log probability of the teacher's favourite token."""
        forward(r)
        lp, best = torch.empty(T, device=device), t_ids[r, :, 0].contiguous()
        dpz.lm_logprobs(logits, best, lp)
        return float(lp.mean())

    before = score(0)
    losses = []
    for step in range(1, steps + 1):
        total = 0.0
        for r in range(N):
            E = forward(r)
            dE = grads[r, :V * D].view(V, D)
            dpz.lm_distill_step(logits, t_ids[r], t_logits[r], weight, loss, logits,
                                temperature=temperature)
            torch.matmul(logits.T, h / D, out=dE)
            torch.matmul(logits, E / D, out=dh)
            dpz.lm_embedding_grad(dh, ids[r], dE, emb_ws, base=dE, scale=scale)
            total += float(loss.mean()) / N
        losses.append(total)
        cfg = dpz.make_cfg(lr=5e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=step,
                           clip_norm=1.0)
        dpz.dp_zero1_step(grads, master, m, v, weights, N, cfg, ws=ws, norm_out=norm)
    return losses, weights[:, :V * D].view(N, V, D), before, score(0)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--width", type=int, default=128)
    ap.add_argument("--ranks", type=int, default=4)
    a = ap.parse_args()
    losses, _, before, after = train(a.steps, a.vocab, a.width, ranks=a.ranks)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i + 1:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses):4d}  loss {losses[-1]:.4f}")
    print(f"mean log probability of the teacher's favourite tokens: {before:.3f} -> {after:.3f}")


if __name__ == "__main__":
    main()
