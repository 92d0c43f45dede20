"""Parameters and gradients that the kernels change in place, and autograd's graphs of them."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build, train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def test_a_step_between_forward_and_backward():
    """The norm's gamma is saved for its gradient: after a step the graph is refused."""
    gamma = torch.nn.Parameter(torch.ones(64, device="cuda"))
    x = torch.randn(5, 64, device="cuda", requires_grad=True)
    opt = train.AdamW([gamma], lr=0.1)
    train.rms_norm(x, gamma).sum().backward(retain_graph=True)
    y = train.rms_norm(x, gamma).sum()
    opt.step()
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    train.rms_norm(x, gamma).sum().backward()


@pytest.mark.parametrize("strided", [False, True])
def test_clipping_between_forward_and_backward(strided):
    """A graph that saved a gradient is refused once that is scaled."""
    p = torch.nn.Parameter(torch.ones(6, 4, device="cuda"))
    p.grad = torch.full((4, 6), 3.0, device="cuda").t() if strided else torch.full((6, 4), 3.0, device="cuda")
    w = torch.ones(6, 4, device="cuda", requires_grad=True)
    loss = (w * p.grad).sum()
    train.clip_grad_norm_([p], 0.5)
    assert abs(float(p.grad.norm()) - 0.5) < 1e-5
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_loaded_after_the_optimizer(bits):
    """As if the optimizer were made after them; in a captured step too, which reads them once more at every replay."""
    def model(seed):
        return [torch.nn.Parameter(torch.randn(n, generator=torch.Generator("cuda").manual_seed(seed + n), device="cuda").bfloat16())
                for n in (5000, 33)]

    def grads(params):
        for p in params:
            p.grad = torch.full_like(p, 0.25)

    late, other = model(1), model(0)
    a, b = (train.AdamW(p, lr=1e-2, state_bits=bits) for p in (late, other))
    with torch.no_grad():
        for p, q in zip(other, late):
            p.copy_(q)
    for params, opt in ((late, a), (other, b)):
        grads(params)
        for _ in range(3):
            opt.step()
    assert all(torch.equal(p, q) for p, q in zip(late, other))
    assert all(torch.equal(s["master"], t["master"]) for s, t in zip(a.state, b.state))


def test_a_captured_step_after_a_change():
    p = torch.nn.Parameter(torch.full((300,), 2.0, device="cuda", dtype=torch.bfloat16))
    p.grad = torch.zeros_like(p)
    opt = train.AdamW([p], lr=0.0, weight_decay=0.0, capturable=True)
    opt.step()
    with torch.no_grad():
        p.fill_(3.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    graph.replay()
    assert bool((p == 3.0).all()) and bool((opt.state[0]["master"] == 3.0).all())
    p.data.fill_(4.0)           # unseen: the masters are as they were
    opt.read_parameters()
    graph.replay()
    assert bool((p == 4.0).all())
