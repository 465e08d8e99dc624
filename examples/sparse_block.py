"""Train a small sparse-expert model through the sharded optimizer.

Every block sends its normalised input to two of its experts and adds the
normalised, gated sum of their answers to the residual stream:

    ids, weights = router(n)
    y  = combine(experts(dispatch(n)))          (zero_expert_*)
    x, n = x + s g norm(y), norm of that         (zero_block_join)

ZeroEngine reduces the ranks' gradients while backward runs; their global norm
is clipped (zero_clip_grad_norm) before the sharded AdamW step.

    python examples/sparse_block.py [--steps 60]
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
    """topk of n_experts two-layer networks for every token."""

    def __init__(self, hidden, inner, n_experts, topk):
        super().__init__()
        self.topk, self.n_experts = topk, n_experts
        self.router = torch.nn.Parameter(torch.randn(n_experts, hidden) / math.sqrt(hidden))
        self.w_in = torch.nn.Parameter(torch.randn(n_experts, hidden, inner) / math.sqrt(hidden))
        self.w_out = torch.nn.Parameter(torch.randn(n_experts, inner, hidden) / math.sqrt(inner))

    def forward(self, n):
        score = torch.softmax((n @ self.router.t()).float(), dim=-1)
        weights, ids = score.topk(self.topk, dim=-1)
        weights = weights / weights.sum(dim=-1, keepdim=True)
        order = Z.zero_expert_sort(ids, self.n_experts)
        xs = Z.expert_dispatch(n, order)
        starts = order.offsets.tolist()
        parts = [torch.nn.functional.gelu(xs[a:b] @ self.w_in[e]) @ self.w_out[e]
                 for e, (a, b) in enumerate(zip(starts, starts[1:]))]
        return Z.expert_combine(torch.cat(parts), weights, order)


class SparseModel(torch.nn.Module):
    def __init__(self, width, hidden, inner, out, blocks=2, n_experts=8, topk=2):
        super().__init__()
        self.scale = 1.0 / math.sqrt(2.0 * blocks)
        self.lift = torch.nn.Linear(width, hidden)
        self.blocks = torch.nn.ModuleList(Experts(hidden, inner, n_experts, topk)
                                          for _ in range(blocks))
        ones = [torch.nn.Parameter(torch.ones(hidden)) for _ in range(3 * blocks + 1)]
        self.w_pre = torch.nn.ParameterList(ones[:blocks + 1])   # before each block, and the head
        self.w_post = torch.nn.ParameterList(ones[blocks + 1:2 * blocks + 1])
        self.gate = torch.nn.ParameterList(ones[2 * blocks + 1:])
        self.head = torch.nn.Linear(hidden, out)

    def forward(self, tokens):
        x = self.lift(tokens)
        x, n = Z.block_join(x, w_pre=self.w_pre[0])
        for k, block in enumerate(self.blocks):
            x, n = Z.block_join(x, block(n), w_post=self.w_post[k], gate=self.gate[k],
                                w_pre=self.w_pre[k + 1], scale=self.scale)
        return self.head(n)


def train(steps=60, ranks=2, tokens=256, seed=0, max_norm=1.0, say=print, **sizes):
    """The losses and gradient norms of every step."""
    shape = dict(width=32, hidden=128, inner=256, out=8) | sizes
    torch.manual_seed(seed)
    model = SparseModel(**shape).to("cuda", torch.bfloat16)
    teacher = torch.nn.Sequential(torch.nn.Linear(shape["width"], 64), torch.nn.Tanh(),
                                  torch.nn.Linear(64, shape["out"])).to("cuda")
    engine = ZeroEngine(model.parameters(), ranks, hparams=Z.AdamW(lr=2e-3))
    history = []
    for t in range(steps):
        mean = 0.0
        for q in range(ranks):
            gen = torch.Generator(device="cuda").manual_seed(1_000_003 * t + q)
            batch = torch.randn(tokens, shape["width"], device="cuda", generator=gen)
            with torch.no_grad():
                want = teacher(batch)
            loss = (model(batch.to(torch.bfloat16)).float() - want).square().mean()
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
