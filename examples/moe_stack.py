"""Trains a stack of Mixture-of-Experts blocks on synthetic data.

    python examples/moe_stack.py [--tokens 512 --hidden 256 --inter 128 --experts 32 --topk 4 --blocks 2 --steps 20]

RMS norm with the residual's addition, the choice of experts (sigmoid scores,
groups, a bias for balance), the sort of the routes, dispatch, the experts'
products, combine, the gradients' norm and AdamW (states in 8 bits, gradients
clipped on the way) are the library's kernels, forward and backward; the gate's
product and SwiGLU are torch.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_mixture_experts_router_gb300 import api, train  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, H, I, E, K, rule):
        super().__init__()
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.E, self.K, self.rule = E, K, rule
        self.gamma = torch.nn.Parameter(torch.ones(H, device="cuda"))
        self.gate = torch.nn.Parameter(torch.randn(E, H, device="cuda") * H ** -0.5)
        self.w1 = torch.nn.Parameter(torch.randn(E, 2 * I, H, **bf) * H ** -0.5)
        self.w2 = torch.nn.Parameter(torch.randn(E, H, I, **bf) * I ** -0.5)
        self.register_buffer("bias", torch.zeros(E, device="cuda"))

    def forward(self, x, residual):
        """The block's output and the residual stream before it: their sum is the next one's input."""
        y, h = train.rms_norm(x, self.gamma, residual)
        ids, w = train.route(y.float() @ self.gate.t(), self.K, self.bias, self.rule)
        routes = self.routes = train.sort_routes(ids, self.E)
        gate, up = train.expert_linear(train.dispatch(y, routes), self.w1, routes).chunk(2, dim=1)
        o = train.expert_linear(F.silu(gate) * up, self.w2, routes)
        return train.combine(o, routes, w), h

    def balance(self, rate):
        """Experts with more than their share of the routes are chosen less."""
        count = self.routes.count.float()
        self.bias -= rate * torch.sign(count - count.mean())


class Stack(torch.nn.Module):
    def __init__(self, H, I, E, K, blocks, rule):
        super().__init__()
        self.blocks = torch.nn.ModuleList(Block(H, I, E, K, rule) for _ in range(blocks))
        self.gamma = torch.nn.Parameter(torch.ones(H, device="cuda"))

    def forward(self, x):
        residual = torch.zeros_like(x)
        for block in self.blocks:
            x, residual = block(x, residual)
        return train.rms_norm(x, self.gamma, residual)[0]


def train_stack(tokens=512, hidden=256, inter=128, experts=32, topk=4, blocks=2, steps=20, lr=3e-3, max_norm=1.0, seed=0):
    """AdamW on the mean squared error to a fixed random target; returns each step's loss, gradient norm and the
    largest share of the routes that one expert has."""
    torch.manual_seed(seed)
    rule = api.RouteRule(score=api.MOE_SCORE_SIGMOID, groups=4, topk_groups=2, group_score=api.MOE_GROUP_TOP2)
    model = Stack(hidden, inter, experts, topk, blocks, rule)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    target = torch.tanh(x.float() @ torch.randn(hidden, hidden, device="cuda") * hidden ** -0.5)
    opt = train.AdamW(model.parameters(), lr=lr, betas=(0.9, 0.95), state_bits=8)
    seen = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (model(x).float() - target).square().mean()
        loss.backward()
        norm = train.grad_norm(model.parameters())
        opt.step(norm=norm, max_norm=max_norm)
        for block in model.blocks:
            block.balance(0.01)
        share = max(float(b.routes.count.max()) for b in model.blocks) / (tokens * topk)
        seen.append((float(loss.detach()), float(norm), share))
        model.blocks[0].routes.check()
    return seen


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, default in (("tokens", 512), ("hidden", 256), ("inter", 128), ("experts", 32), ("topk", 4), ("blocks", 2),
                          ("steps", 20)):
        p.add_argument("--" + name, type=int, default=default)
    for i, (loss, norm, share) in enumerate(train_stack(**vars(p.parse_args()))):
        print(f"step {i:3d}  loss {loss:.5f}  gradient norm {norm:.4f}  largest share {share:.3f}")
