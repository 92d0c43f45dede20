"""Trains one pre-norm Mixture-of-Experts block on synthetic data.

    python examples/moe_block.py [--tokens 512 --hidden 256 --inter 128 --experts 8 --topk 2 --steps 20]

Layer norm, the sort of the routes, dispatch, the experts' products, combine
and the gradient clipping are the library's kernels, forward and backward; the
router (a torch product, softmax and top-K), SwiGLU and the optimizer are torch.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_mixture_experts_router_gb300 import train  # noqa: E402


class MoEBlock(torch.nn.Module):
    def __init__(self, H, I, E, K):
        super().__init__()
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.E, self.K = E, K
        self.gamma = torch.nn.Parameter(torch.ones(H, device="cuda"))
        self.beta = torch.nn.Parameter(torch.zeros(H, device="cuda"))
        self.gate = torch.nn.Parameter(torch.randn(E, H, device="cuda") * H ** -0.5)
        self.w1 = torch.nn.Parameter(torch.randn(E, 2 * I, H, **bf) * H ** -0.5)
        self.w2 = torch.nn.Parameter(torch.randn(E, H, I, **bf) * I ** -0.5)

    def route(self, h):
        """Top-K experts of h [T, H] and their weights (softmax over the selected)."""
        logits = h.float() @ self.gate.t()
        top, ids = logits.topk(self.K, dim=1)
        return ids.to(torch.int32), torch.softmax(top, dim=1)

    def forward(self, x):
        h = train.layer_norm(x, self.gamma, self.beta)
        ids, w = self.route(h)
        routes = self.routes = train.sort_routes(ids, self.E)
        z = train.expert_linear(train.dispatch(h, routes), self.w1, routes)
        gate, up = z.chunk(2, dim=1)
        o = train.expert_linear(F.silu(gate) * up, self.w2, routes)
        return x + train.combine(o, routes, w)


def train_block(tokens=512, hidden=256, inter=128, experts=8, topk=2, steps=20, lr=1.0, max_norm=0.1, seed=0):
    """SGD on the mean squared error to a fixed random target; returns each step's loss and gradient norm."""
    torch.manual_seed(seed)
    block = MoEBlock(hidden, inter, experts, topk)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    target = x + 0.5 * torch.tanh(x.float() @ torch.randn(hidden, hidden, device="cuda") * hidden ** -0.5).bfloat16()
    opt = torch.optim.SGD(block.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = (block(x).float() - target.float()).square().mean()
        loss.backward()
        norm = train.clip_grad_norm_(block.parameters(), max_norm)
        opt.step()
        losses.append((float(loss.detach()), float(norm)))
        block.routes.check()        # errors found on the device (it waits, as the two reads before it do)
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, default in (("tokens", 512), ("hidden", 256), ("inter", 128), ("experts", 8), ("topk", 2), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=default)
    for i, (loss, norm) in enumerate(train_block(**vars(p.parse_args()))):
        print(f"step {i:3d}  loss {loss:.5f}  gradient norm {norm:.4f}")
