"""Training a draft model on what the target model says, end to end: random
models, one GPU, the calls on rows of logits.

    python examples/draft_training.py [--steps 50] [--rows 512] [--top 32]

The target's rows are seen once: token_logprobs keeps their likeliest tokens
and log probabilities (the record, a hundredth of the logits' bytes).  Then
each step
  distill_grad         the draft's divergence from the record and its gradient
                       in the logits, from which autograd goes on into the model
and, for tokens that were emitted rather than recorded,
  token_logprobs       their log probabilities under the draft, and entropies
  token_logprobs_grad  the gradient of the mean of both
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from spec_verify_gb300 import binding, scores  # noqa: E402


class Draft(torch.nn.Module):
    """Logits by the last token alone; random weights."""

    def __init__(self, vocab=2000, hidden=64, dtype=torch.bfloat16, seed=0):
        super().__init__()
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.nn.Parameter(torch.randn(*s, generator=g, device="cuda"))  # noqa: E731
        self.embed, self.head, self.dtype = rand(vocab, hidden), rand(hidden, vocab), dtype

    def forward(self, tokens):
        hidden = self.embed[tokens] * self.embed.shape[1] ** -0.5
        return (hidden @ self.head).to(self.dtype)


def checked(status):
    flags = int(status)
    if flags:
        raise RuntimeError("a token past the vocabulary" if flags & binding.ROW_BAD_TOKEN else "flags %d" % flags)


def distill(model, tokens, record, temperature=1.0):
    """The gradients of the mean divergence into the model's parameters.
    Returns (losses [rows], logits, their gradient)."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    logits = model(tokens)
    weight = torch.full((len(tokens),), 1.0 / len(tokens), device="cuda")
    loss, grad = scores.distill_grad(logits.detach(), record.top_ids, record.top_logprobs, weight, tail=True,
                                     temperature=temperature, status=status)
    checked(status)
    logits.backward(grad)
    return loss, logits.detach(), grad


def follow(model, tokens, emitted, bonus=0.01):
    """The gradients of the mean of -ln p(emitted) - bonus * entropy (negative
    emitted ids: padding).  Returns (that mean, logits, their gradient)."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    logits = model(tokens)
    live = (emitted >= 0).float()
    n = live.sum().clamp_min(1)
    got = scores.token_logprobs(logits.detach(), emitted[:, None], entropy=True, status=status)
    checked(status)
    grad = scores.token_logprobs_grad(logits.detach(), emitted[:, None], (-live / n)[:, None], -bonus * live / n)
    logits.backward(grad)
    return -((got.logprobs[:, 0] + bonus * got.entropy) * live).sum() / n, logits.detach(), grad


def acceptance(target, draft):
    """Chance that a draft is accepted: sum over tokens of min(p, q), the mean over rows."""
    return torch.minimum(target.float().softmax(-1), draft.float().softmax(-1)).sum(-1).mean()


def main():
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=50)
    parser.add_argument("--rows", type=int, default=512)
    parser.add_argument("--top", type=int, default=32)
    args = parser.parse_args()
    target, draft = Draft(hidden=96, seed=1), Draft(seed=2)
    g = torch.Generator("cuda").manual_seed(3)
    tokens = torch.randint(0, 2000, (args.rows,), generator=g, device="cuda")
    with torch.no_grad():
        wanted = target(tokens) * 3
        record = scores.token_logprobs(wanted, top=args.top)
        emitted = torch.multinomial(wanted.float().softmax(-1), 1, generator=g)[:, 0].int()
        before = acceptance(wanted, draft(tokens))
    optimizer = torch.optim.Adam(draft.parameters(), lr=0.05)
    for step in range(args.steps):
        optimizer.zero_grad()
        loss, _, _ = distill(draft, tokens, record)
        value, _, _ = follow(draft, tokens, emitted)
        optimizer.step()
        if step % 10 == 0 or step + 1 == args.steps:
            print("step %d: divergence %.3f, emitted tokens %.3f" % (step, loss.mean().item(), value.item()))
    with torch.no_grad():
        print("accepted drafts: %.3f, before %.3f" % (acceptance(wanted, draft(tokens)).item(), before.item()))


if __name__ == "__main__":
    main()
