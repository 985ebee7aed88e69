"""A student with routed experts learns from a teacher's stored top logits.

    python examples/distill_moe.py [steps]

The teacher runs once; segmented_row_topk keeps the top of every row of its
logits (values, columns) and the row's log-sum-exp.  Each training step routes
the tokens with segmented_row_topk on the router's logits, adds
expert_balance_loss, which evens the experts' load, to topk_distill_loss, which
pulls the student towards the teacher, and follows their gradients.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lsd_radix_sort_amd as lrs  # noqa: E402

VOCAB, WIDTH, EXPERTS, CHOSEN, TOP, TOKENS = 5003, 64, 16, 2, 24, 512


class Student(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.router = torch.nn.Linear(WIDTH, EXPERTS, bias=False)
        self.up = torch.nn.Parameter(torch.randn(EXPERTS, WIDTH, 2 * WIDTH) * 0.1)
        self.down = torch.nn.Parameter(torch.randn(EXPERTS, 2 * WIDTH, WIDTH) * 0.1)
        self.head = torch.nn.Linear(WIDTH, VOCAB, bias=False)

    def forward(self, x):
        scores = self.router(x)
        _, experts = lrs.segmented_row_topk(scores.detach(), CHOSEN)
        # its values carry no gradient; the scores gathered at the chosen experts do
        share = torch.softmax(torch.gather(scores, 1, experts), dim=1)
        y = x
        for e in range(EXPERTS):
            token, slot = torch.nonzero(experts == e, as_tuple=True)
            out = torch.relu(x[token] @ self.up[e]) @ self.down[e]
            y = y.index_add(0, token, out * share[token, slot, None])
        return self.head(y), scores, experts


def main(steps: int = 60, seed: int = 0):
    """Trains for `steps` steps; returns the distillation loss and the largest expert's share of the
    slots, both by step."""
    torch.manual_seed(seed)
    dev = torch.device("cuda")
    x = torch.randn(TOKENS, WIDTH, device=dev)
    teacher = 2.0 * torch.randn(VOCAB, WIDTH, device=dev) / WIDTH ** 0.5
    logits = x @ teacher.T
    values, columns = lrs.segmented_row_topk(logits, TOP)
    lse = torch.logsumexp(logits.double(), dim=1).float()
    weights = torch.full((TOKENS,), 1.0 / TOKENS, device=dev)
    weights[-TOKENS // 16:] = 0.0  # padding tokens
    counted = weights > 0

    student = Student().to(dev)
    adam = torch.optim.Adam(student.parameters(), lr=3e-3)
    losses, shares = [], []
    for _ in range(steps):
        out, scores, experts = student(x)
        distill = lrs.topk_distill_loss(out, values, columns, teacher_lse=lse, row_weights=weights)
        balance, counts = lrs.expert_balance_loss(scores, experts, balance_weight=0.05, z_weight=1e-3, row_mask=counted)
        adam.zero_grad()
        (distill + balance).backward()
        adam.step()
        losses.append(float(distill.detach()))
        shares.append(float(counts.max()) / float(counts.sum()))
    return losses, shares


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 60
    losses, shares = main(steps)
    for i in range(0, steps, max(1, steps // 10)):
        print(f"step {i:4d}  distillation loss {losses[i]:.4f}  largest expert {100 * shares[i]:.1f}% of the slots")
    print(f"last       distillation loss {losses[-1]:.4f}  largest expert {100 * shares[-1]:.1f}% of the slots")
