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
