"""The training operators together: one Mixture-of-Experts block, forward and
backward, against the same block in 64-bit torch.

Bound: the block rounds to BF16 after the layer norm, the two products, SwiGLU
and the sum (half an ulp is 2^-8, about 2^-9.5 in the mean square), and its
gradient after as many steps again; each rounding enters a result once, so a
result's relative error in the 2-norm stays below the sum of the half ulps:
6 * 2^-8 forward, 12 * 2^-8 for a gradient."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

from nvfp4_mixture_experts_router_gb300 import api, build, train

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def reference(block, x, ids):
    """The block in 64 bits on the same routes; returns its output and parameters."""
    p = {n: v.detach().double().requires_grad_(True) for n, v in block.named_parameters()}
    x = x.detach().double().requires_grad_(True)
    h = F.layer_norm(x, (x.shape[1],), p["gamma"], p["beta"], 1e-5)
    logits = h @ p["gate"].t()
    w = torch.softmax(logits.gather(1, ids.long()), dim=1)
    z = torch.einsum("th,tknh->tkn", h, p["w1"][ids.long()])
    g, u = z.chunk(2, dim=2)
    o = torch.einsum("tki,tkhi->tkh", F.silu(g) * u, p["w2"][ids.long()])
    return x + (o * w[..., None]).sum(1), x, p


@pytest.mark.parametrize("T,H,I,E,K", [(1, 64, 32, 4, 2), (33, 64, 40, 16, 3), (200, 256, 128, 8, 2)])
def test_block_against_64_bits(T, H, I, E, K):
    torch.manual_seed(T)
    block = moe_block.MoEBlock(H, I, E, K)
    x = torch.randn(T, H, device="cuda").bfloat16().requires_grad_(True)
    ids, _ = block.route(train.layer_norm(x, block.gamma, block.beta))
    y = block(x)
    want, x64, p64 = reference(block, x, ids)
    c = torch.randn(T, H, device="cuda").bfloat16()
    y.backward(c)
    want.backward(c.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(y.detach(), want.detach()) < 6 * 2.0 ** -8
    assert rel(x.grad, x64.grad) < 12 * 2.0 ** -8
    for n, v in block.named_parameters():
        assert rel(v.grad, p64[n].grad) < 12 * 2.0 ** -8, n


def test_block_with_dropped_routes():
    """Routes dropped by a capacity limit give nothing, and no gradient."""
    torch.manual_seed(5)
    T, H, N, E, K = 40, 64, 96, 5, 3
    ids = torch.randint(0, E, (T, K), device="cuda", dtype=torch.int32)
    ids[torch.rand(T, K, device="cuda") < 0.3] = -1
    x = torch.randn(T, H, device="cuda").bfloat16().requires_grad_(True)
    w = (torch.randn(E, N, H, device="cuda") * H ** -0.5).bfloat16().requires_grad_(True)
    s = torch.rand(T, K, device="cuda").requires_grad_(True)
    routes = train.sort_routes(ids, E)
    y = train.combine(train.expert_linear(train.dispatch(x, routes), w, routes), routes, s)
    c = torch.randn(T, N, device="cuda").bfloat16()
    y.backward(c)
    x2, w2, s2 = (v.detach().double().requires_grad_(True) for v in (x, w, s))
    o = torch.einsum("th,tknh->tkn", x2, w2[ids.clamp(min=0).long()])
    want = (o * torch.where(ids >= 0, s2, 0.0)[..., None]).sum(1)
    want.backward(c.double())
    for a, b in ((y.detach(), want.detach()), (x.grad, x2.grad), (w.grad, w2.grad), (s.grad, s2.grad)):
        assert float((a.double() - b).norm() / b.norm()) < 4 * 2.0 ** -8
    assert not s.grad[ids < 0].any()


def test_example_descends():
    """Gradient descent on one batch with clipped steps: the loss falls at
    every step, and the gradients' norms are above the limit (clipping acts)."""
    steps = moe_block.train_block(steps=8, max_norm=0.05)
    losses = [l for l, _ in steps]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert all(n > 0.05 for _, n in steps)


def test_clip_grad_norm():
    p = [torch.nn.Parameter(torch.zeros(n, device="cuda", dtype=d)) for n, d in ((10, torch.float32), (7, torch.bfloat16))]
    assert float(train.clip_grad_norm_(p, 1.0)) == 0.0
    p[0].grad, p[1].grad = torch.full((10,), 3.0, device="cuda"), torch.full((7,), 2.0, device="cuda").bfloat16()
    norm = float(train.clip_grad_norm_(p, 1.0))
    assert abs(norm - (90.0 + 28.0) ** 0.5) < 1e-5
    total = (p[0].grad.double().square().sum() + p[1].grad.double().square().sum()).sqrt()
    assert abs(float(total) - 1.0) < 2.0 ** -8
