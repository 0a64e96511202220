"""A small distillation run with the library's operators: teacher and student are a layer norm,
a SwiGLU gate and a projection to a vocabulary each; the teacher's top log probabilities are
kept once, the student learns from them.

    python -m workloads.distill --steps 20

Weights and inputs are random (seeded).  Prints the loss, and the student's mean log
probability of the teacher's first choice, before and after.
"""
from __future__ import annotations

import argparse

import torch

import swish_activation_backward_amd as swg
from swish_activation_backward_amd.autograd import LayerNorm, SwiGLU, distill_loss, token_logprobs


class Head(torch.nn.Module):
    def __init__(self, width, hidden, vocab, device, dtype):
        super().__init__()
        self.norm = LayerNorm(width, device=device)
        self.gate = SwiGLU(width, hidden, device=device, dtype=dtype)
        self.out = torch.nn.Parameter(
            torch.randn(hidden, vocab, device=device, dtype=dtype) * (2.0 / hidden ** 0.5))

    def forward(self, x):
        return self.gate(self.norm(x)) @ self.out


def run(steps=20, tokens=512, width=256, hidden=512, vocab=8192, top=32, temperature=2.0,
        dtype=torch.bfloat16, seed=0, lr=0.5):
    """Returns the mean loss of every step and the student's mean log probability of the
    teacher's first choice before and after."""
    device = torch.device("cuda")
    torch.manual_seed(seed)
    teacher, student = (Head(width, hidden, vocab, device, dtype) for _ in range(2))
    x = torch.randn(tokens, width, device=device, dtype=dtype)
    with torch.no_grad():
        kept = swg.token_logprobs(teacher(x), top=top)
    first = kept.top_id[:, 0].contiguous()

    def agreement():
        with torch.no_grad():
            return token_logprobs(student(x), first)[0].mean().item()

    opt = torch.optim.AdamW(student.parameters(), lr=lr * 1e-2)
    before, losses = agreement(), []
    for _ in range(steps):
        opt.zero_grad()
        loss = distill_loss(student(x), kept.top_logprob, kept.top_id, temperature).mean()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), before, agreement()


def train_step_in_one_pass(student, x, kept, temperature):
    """One step's loss and gradients with loss and logit gradient from a single pass over the
    logits (the row weights, 1 / rows, are known beforehand)."""
    logits = student(x)
    weight = torch.full((x.shape[0],), 1.0 / x.shape[0], device=x.device)
    loss, _, dlogits = swg.distill_fwd_bwd(logits.detach(), kept.top_logprob, kept.top_id, weight,
                                           temperature=temperature)
    logits.backward(dlogits)
    return loss.mean()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=8192)
    args = ap.parse_args()
    losses, before, after = run(args.steps, args.tokens, vocab=args.vocab)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; log probability of the teacher's first "
          f"choice {before:.3f} -> {after:.3f}")


if __name__ == "__main__":
    main()
