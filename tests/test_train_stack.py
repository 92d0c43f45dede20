"""Routing, RMS norm and AdamW with the other training operators, as they are
used: a stack of blocks, forward and backward, against the same stack in 64-bit
torch, and the optimizer's step after it.

Bound: a block rounds to BF16 after the norm, its residual's sum, the two
products, SwiGLU and the sum (half an ulp is 2^-8), and its gradient after as
many steps again; each rounding enters a result once a block, so a result's
relative error in the 2-norm stays below the sum of the half ulps: 7 * 2^-8 a
block forward, 14 * 2^-8 a block for a gradient."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

from nvfp4_mixture_experts_router_gb300 import api, build, train

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_stack  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def reference(model, x, ids, rule, K):
    """The stack in 64 bits on the same routes."""
    p = {n: v.detach().double().requires_grad_(True) for n, v in model.named_parameters()}
    x = x.detach().double().requires_grad_(True)
    norm = lambda v, g: v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * g      # noqa: E731
    h = x
    for i, e in enumerate(ids):
        q = {n: p[f"blocks.{i}.{n}"] for n in ("gamma", "gate", "w1", "w2")}
        y = norm(h, q["gamma"])
        l = (y @ q["gate"].t()).gather(1, e.long())
        s = torch.sigmoid(l) if rule.score == api.MOE_SCORE_SIGMOID else torch.exp(l)
        w = rule.scale * s / s.sum(1, keepdim=True)
        g, u = torch.einsum("th,tknh->tkn", y, q["w1"][e.long()]).chunk(2, dim=2)
        h = h + (torch.einsum("tki,tkhi->tkh", F.silu(g) * u, q["w2"][e.long()]) * w[..., None]).sum(1)
    return norm(h, p["gamma"]), x, p


@pytest.mark.parametrize("T,H,I,E,K,blocks", [(1, 64, 32, 8, 2, 1), (37, 64, 40, 16, 3, 2), (200, 256, 128, 32, 4, 2)])
@pytest.mark.parametrize("score", [api.MOE_SCORE_SIGMOID, api.MOE_SCORE_SOFTMAX])
def test_stack_against_64_bits(T, H, I, E, K, blocks, score):
    torch.manual_seed(T)
    rule = api.RouteRule(score=score, groups=4, topk_groups=2, group_score=api.MOE_GROUP_TOP2, scale=1.5)
    model = moe_stack.Stack(H, I, E, K, blocks, rule)
    for b in model.blocks:
        b.bias += 0.02 * torch.randn(E, device="cuda")
    seen = []
    route = train.route
    train.route = lambda *a: seen.append(route(*a)) or seen[-1]
    try:
        x = torch.randn(T, H, device="cuda").bfloat16().requires_grad_(True)
        y = model(x)
    finally:
        train.route = route
    want, x64, p64 = reference(model, x, [ids for ids, _ in seen], rule, K)
    c = torch.randn(T, H, device="cuda").bfloat16()
    y.backward(c)
    want.backward(c.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())      # noqa: E731
    assert rel(y.detach(), want.detach()) < 7 * blocks * 2.0 ** -8
    assert rel(x.grad, x64.grad) < 14 * blocks * 2.0 ** -8
    for n, v in model.named_parameters():
        assert rel(v.grad, p64[n].grad) < 14 * blocks * 2.0 ** -8, n
    for b, (ids, w) in zip(model.blocks, seen):
        assert bool(((ids >= 0) & (ids < E)).all()) and bool(((w.sum(1) - 1.5).abs() < 1e-5).all())
        b.routes.check()
    # a step: each parameter moves by lr at most (times 1 + decay), and the norm is that of all gradients
    norm = train.grad_norm(model.parameters())
    total = torch.cat([v.grad.double().reshape(-1) for v in model.parameters()]).norm()
    assert abs(float(norm) - float(total)) <= 1e-5 * float(total)
    before = {n: v.detach().clone().float() for n, v in model.named_parameters()}
    opt = train.AdamW(model.parameters(), lr=1e-3, weight_decay=0.0, state_bits=8)
    opt.step(norm=norm)
    for n, v in model.named_parameters():
        # the first step is lr * sign(g) but for eps; BF16 parameters round, by 2^-8 of the new value, which is the
        # old one and the step at most
        moved = (v.detach().float() - before[n]).abs()
        assert bool((moved <= 1.001e-3 + 2.0 ** -8 * (before[n].abs() + 1.001e-3) + 1e-7).all()), n
        assert bool((moved > 0).any()), n


def test_the_example_runs():
    seen = moe_stack.train_stack(tokens=100, hidden=64, inter=32, experts=16, topk=2, steps=3)
    assert len(seen) == 3 and all(0 < n < float("inf") and l == l for l, n, _ in seen)


def test_a_step_in_a_graph():
    """Norm, routing, their gradients, the gradients' norm and AdamW captured together and replayed: the same bits
    as one by one."""
    T, H, E, K = 64, 256, 32, 4
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
    x, res, w, gamma = r(T, H).bfloat16(), r(T, H).bfloat16(), r(E, H) * 0.1, torch.ones(H, device="cuda")
    rule = api.RouteRule(score=api.MOE_SCORE_SIGMOID)

    def build_all():
        p = [torch.nn.Parameter(w.clone()), torch.nn.Parameter(gamma.clone())]
        for q in p:
            q.grad = torch.zeros_like(q)
        return p, train.AdamW(p, lr=1e-2, capturable=True)

    def step(p, opt):
        y, h = train.rms_norm(x, p[1], res)
        _, weights = train.route(y.float() @ p[0].t(), K, None, rule)
        loss = (weights * target).sum() + h.float().mean()
        for q, d in zip(p, torch.autograd.grad(loss, p)):
            q.grad.copy_(d)
        opt.step(norm=train.grad_norm(p), max_norm=0.1)

    target = r(T, K)
    a, oa = build_all()
    b, ob = build_all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for p, o in ((a, oa), (b, ob)):
            step(p, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, oa)
    for _ in range(3):
        graph.replay()
        step(b, ob)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T", [0, 1, 5])
def test_gradients_of_plain_sums(T):
    """A sum's gradient is one broadcast number: without tokens its strides are 0 still."""
    H = 40
    x, r = (torch.randn(T, H, device="cuda", requires_grad=True) for _ in range(2))
    gamma = torch.randn(H, device="cuda", requires_grad=True)
    beta = torch.zeros(H, device="cuda", requires_grad=True)
    y, h = train.rms_norm(x, gamma, r)
    (y.sum() + h.sum()).backward()
    train.layer_norm(x, gamma, beta).sum().backward()
    logits = torch.randn(T, 6, device="cuda", requires_grad=True)
    train.route(logits, 2)[1].sum().backward()
    for t in (x, r, gamma, beta, logits):
        assert t.grad.shape == t.shape and bool(t.grad.isfinite().all())
    # beta's gradient is T, whatever x is
    assert torch.equal(beta.grad, torch.full_like(beta, float(T)))
