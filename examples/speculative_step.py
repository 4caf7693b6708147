"""Speculative decoding over a paged 8-bit cache, end to end: a small target
model of random weights, a draft model that knows the last token alone, and
the five calls of a step on one GPU.

    python examples/speculative_step.py [--steps 20] [--batch 8] [--drafts 4]

One step of every request adds the token it emitted last and K drafts:
  block_plan          places in the cache for the step's tokens
  qk_norm_rope        norm and rotation of queries and keys, in place in the
                      fused projection
  cache_append        keys and values into the cache, in 8 bits
  cache_attention     the queries over the cache
  spec_verify_probs   the check of the drafts: 1 to K + 1 new tokens
The rejected drafts stay in the cache past the request's length, where the
next step writes over them.  Lengths, block table and tokens stay on the
device; only the plan's status word is read back in a step, since a request
that found no blocks has no rows in what follows.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from spec_verify_gb300 import binding, cache  # noqa: E402


class Target:
    """`layers` layers of attention over a cache, between an embedding and a
    head; random weights."""

    def __init__(self, vocab=2000, hidden=256, layers=2, heads=8, kv_heads=2, dim=64, blocks=512, block=16,
                 codes=torch.float8_e4m3fn, dtype=torch.bfloat16, max_len=4096, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.vocab, self.heads, self.kv_heads, self.dim, self.block = vocab, heads, kv_heads, dim, block
        self.dtype = dtype
        self.embed = rand(vocab, hidden)
        self.qkv = [(rand(hidden, (heads + 2 * kv_heads) * dim) * hidden ** -0.5).to(dtype) for _ in range(layers)]
        self.out = [(rand(heads * dim, hidden) * (heads * dim) ** -0.5).to(dtype) for _ in range(layers)]
        self.q_weight = [1 + 0.1 * rand(dim) for _ in range(layers)]
        self.k_weight = [1 + 0.1 * rand(dim) for _ in range(layers)]
        self.head = rand(hidden, vocab) * 3 * hidden ** -0.5
        self.caches = [cache.new_cache(blocks, kv_heads, block, dim, codes) for _ in range(layers)]
        self.table = cache.rope_table(max_len, dim)
        self.workspace = None
        self.attended = None          # of the last layer: what its attention read and gave

    def draft(self, tokens):
        """Probabilities of the token after each, by the last token alone."""
        return (self.embed[tokens] @ self.head).softmax(-1)

    def step(self, tokens, plan, block_table):
        """Probabilities [T, vocab] of the token after each of the step's."""
        x = self.embed[tokens]
        n, hq, hk, d = tokens.shape[0], self.heads, self.kv_heads, self.dim
        need = cache.attention_workspace_bytes(n, hq, hk, d, plan.lens.shape[0])
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        for i, kv in enumerate(self.caches):
            normed = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            fused = (normed.to(self.dtype) @ self.qkv[i]).view(n, hq + 2 * hk, d)
            q, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
            cache.qk_norm_rope(q, k, plan.position, self.table, self.q_weight[i], self.k_weight[i], out_q=q, out_k=k)
            cache.cache_append(kv, k, v, plan.slot)
            o = torch.empty(n, hq, d, dtype=self.dtype, device="cuda")
            cache.cache_attention(kv, q, plan.start, plan.lens, block_table, out=o, workspace=self.workspace)
            x = x + (o.view(n, -1) @ self.out[i]).float()
            self.attended = kv, q, plan, block_table, o
        return (x @ self.head).softmax(-1)


def plan_step(model, lens, add, held, free, head, table, tokens):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = cache.block_plan(lens, add, held, free, head, table, model.block, free.shape[0], tokens, status=status)
    flags = int(status)
    if flags:
        raise RuntimeError("the cache has too few blocks" if flags & binding.ROW_NO_CAPACITY else "flags %d" % flags)
    return plan


def generate(model, batch=8, drafts=4, steps=20, prompt=17, seed=1, after_step=None):
    """`steps` steps of `batch` requests from prompts of 1 to `prompt` random
    tokens.  Returns (accepted [steps, batch], ids [steps, batch, drafts + 1],
    lens [batch])."""
    g = torch.Generator("cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    blocks = model.caches[0][0].shape[0]
    held, lens, head = torch.zeros(batch, **i32), torch.zeros(batch, **i32), torch.zeros(1, **i32)
    table = torch.zeros(batch, blocks, **i32)
    free = torch.randperm(blocks, generator=g, device="cuda").int()

    # the prompts, all but their last token: one ragged step
    sizes = [1 + (7 * b + 3) % prompt for b in range(batch)]
    tokens = torch.randint(0, model.vocab, (sum(sizes),), generator=g, device="cuda")
    last = torch.tensor(sizes).cumsum(0).cuda() - 1
    keep = torch.ones(len(tokens), dtype=torch.bool, device="cuda")
    keep[last] = False
    emitted = tokens[last]
    add = torch.tensor([s - 1 for s in sizes], **i32)
    if sum(sizes) > batch:
        plan = plan_step(model, lens, add, held, free, head, table, sum(sizes) - batch)
        model.step(tokens[keep], plan, table)
        lens, held, head = plan.lens, plan.held, plan.free_head

    add = torch.full((batch,), drafts + 1, **i32)
    accepted, ids = [], []
    for _ in range(steps):
        # the draft model proposes, one token after the other
        chain, q = [emitted], []
        for _ in range(drafts):
            q.append(model.draft(chain[-1]))
            chain.append(torch.multinomial(q[-1], 1, generator=g)[:, 0])
        chain = torch.stack(chain, 1)                                     # [batch, drafts + 1]
        plan = plan_step(model, lens, add, held, free, head, table, batch * (drafts + 1))
        p = model.step(chain.view(-1), plan, table).view(batch, drafts + 1, -1)
        noise = torch.empty(batch, model.vocab, device="cuda").exponential_(generator=g).clamp_min_(1e-30)
        uniforms = torch.rand(batch, drafts, generator=g, device="cuda")
        got, out = binding.spec_verify_probs(p, torch.stack(q, 1), chain[:, 1:].int().contiguous(), uniforms, noise)
        if after_step is not None:
            after_step(model, plan)
        # the last token of each row goes first in the next step
        emitted = out.gather(1, got[:, None].long().clamp_min(0))[:, 0].long()
        lens, held, head = lens + got + 1, plan.held, plan.free_head
        accepted.append(got)
        ids.append(out)
    if any(int(got.min()) < 0 for got in accepted):
        raise RuntimeError("a target row without probabilities")
    return torch.stack(accepted), torch.stack(ids), lens


def main():
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=20)
    parser.add_argument("--batch", type=int, default=8)
    parser.add_argument("--drafts", type=int, default=4)
    args = parser.parse_args()
    model = Target(blocks=args.batch * (2 + (32 + (args.steps + 1) * (args.drafts + 1)) // 16))
    accepted, ids, lens = generate(model, args.batch, args.drafts, args.steps)
    print("accepted drafts per step: %.2f of %d" % (accepted.float().mean().item(), args.drafts))
    print("tokens per step: %.2f" % (accepted.float().mean().item() + 1))
    print("lengths: %s" % lens.tolist())
    print("request 0: %s" % [int(t) for row in ids[:, 0].tolist() for t in row if t >= 0])


if __name__ == "__main__":
    main()
