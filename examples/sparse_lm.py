"""Train a small sparse-expert language model through the sharded optimizer.

Token ids in, the loss of the next token out, one table for both ends:

    x = scale table[ids]                                (zero_embedding)
    ids, weights, balance = route(n router^T)           (zero_expert_route)
    y  = combine(experts(dispatch(n)))                  (zero_expert_*)
    x, n = x + s g norm(y), norm of that                (zero_block_join)
    loss = cross entropy of n table^T                   (zero_linear_cross_entropy)

The logits are never in memory; the table takes the gradients of both ends.

    python examples/sparse_lm.py [--steps 60]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_optimizer_flatten_gb300 as Z  # noqa: E402
from zero_sharded_optimizer_flatten_gb300.engine import ZeroEngine  # noqa: E402


class Experts(torch.nn.Module):
    """topk of n_experts two-layer networks for every token, and the losses
    that keep them in balance."""

    def __init__(self, hidden, inner, n_experts, topk):
        super().__init__()
        self.topk, self.n_experts = topk, n_experts
        self.router = torch.nn.Parameter(torch.randn(n_experts, hidden) / math.sqrt(hidden))
        self.w_in = torch.nn.Parameter(torch.randn(n_experts, hidden, inner) / math.sqrt(hidden))
        self.w_out = torch.nn.Parameter(torch.randn(n_experts, inner, hidden) / math.sqrt(inner))

    def forward(self, n):
        ids, weights, _, losses = Z.expert_route(n @ self.router.t(), self.topk)
        order = Z.zero_expert_sort(ids, self.n_experts)
        xs = Z.expert_dispatch(n, order)
        starts = order.offsets.tolist()
        parts = [torch.nn.functional.gelu(xs[a:b] @ self.w_in[e]) @ self.w_out[e]
                 for e, (a, b) in enumerate(zip(starts, starts[1:]))]
        return Z.expert_combine(torch.cat(parts), weights, order), losses


class SparseLM(torch.nn.Module):
    def __init__(self, vocab, hidden, inner, blocks=2, n_experts=8, topk=2):
        super().__init__()
        self.scale = 1.0 / math.sqrt(2.0 * blocks)
        self.hidden = hidden
        self.table = torch.nn.Parameter(torch.randn(vocab, hidden) / math.sqrt(hidden))
        self.blocks = torch.nn.ModuleList(Experts(hidden, inner, n_experts, topk) for _ in range(blocks))
        ones = [torch.nn.Parameter(torch.ones(hidden)) for _ in range(3 * blocks + 1)]
        self.w_pre = torch.nn.ParameterList(ones[:blocks + 1])   # before each block, and the head
        self.w_post = torch.nn.ParameterList(ones[blocks + 1:2 * blocks + 1])
        self.gate = torch.nn.ParameterList(ones[2 * blocks + 1:])

    def forward(self, ids, targets, balance=1e-2, z=1e-3):
        """The mean loss of the targets (-1: none), with the routers' losses."""
        x = Z.embedding(ids.reshape(-1), self.table, scale=math.sqrt(self.hidden))
        extra = 0.0
        x, n = Z.block_join(x, w_pre=self.w_pre[0])
        for k, block in enumerate(self.blocks):
            y, losses = block(n)
            extra = extra + balance * losses[0] + z * losses[1]
            x, n = Z.block_join(x, y, w_post=self.w_post[k], gate=self.gate[k],
                                w_pre=self.w_pre[k + 1], scale=self.scale)
        return Z.linear_cross_entropy(n, self.table, targets.reshape(-1)) + extra


def texts(vocab, count, length, gen):
    """Sequences whose next token is mostly a fixed function of the last one."""
    ids = torch.randint(0, vocab, (count, length + 1), device="cuda", generator=gen)
    for t in range(1, length + 1):
        follows = torch.rand(count, device="cuda", generator=gen) < 0.9
        ids[:, t] = torch.where(follows, (ids[:, t - 1] * 7 + 3) % vocab, ids[:, t])
    return ids[:, :-1], ids[:, 1:]


def train(steps=60, ranks=2, count=8, length=64, seed=0, max_norm=1.0, say=print, **sizes):
    """The losses and gradient norms of every step."""
    shape = dict(vocab=500, hidden=128, inner=256) | sizes
    torch.manual_seed(seed)
    model = SparseLM(**shape).to("cuda", torch.bfloat16)
    engine = ZeroEngine(model.parameters(), ranks, hparams=Z.AdamW(lr=2e-3))
    history = []
    for t in range(steps):
        mean = 0.0
        for q in range(ranks):
            gen = torch.Generator(device="cuda").manual_seed(1_000_003 * t + q)
            ids, targets = texts(shape["vocab"], count, length, gen)
            loss = model(ids, targets)
            engine.backward(loss, q)
            mean += float(loss.detach()) / ranks
        norm = engine.clip_grad_norm(max_norm)
        engine.step()
        history.append((mean, float(norm)))
        if t % 10 == 0 or t + 1 == steps:
            say(f"step {t:4d}  loss {mean:.4f}  gradient norm {history[-1][1]:.4f}")
    engine.remove_hooks()
    return history


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    train(parser.parse_args().steps)
