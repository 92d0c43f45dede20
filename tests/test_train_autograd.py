"""train.py beside the block: what its functions do with dropped routes, row
buffers of another size, odd gradients, and errors found on the device."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build, train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


@pytest.mark.parametrize("norm", [None, torch.zeros(1)])
def test_a_norm_that_is_no_cuda_tensor_is_a_type_error(norm):
    grads = api.GradList([torch.zeros(8, device="cuda")])
    with pytest.raises(TypeError):
        api.moe_nvfp4_grad_norm(grads, norm, torch.zeros(256, device="cuda"))
    with pytest.raises(TypeError):
        api.moe_nvfp4_grad_clip(grads, norm, 1.0)


def param(grad):
    p = torch.nn.Parameter(torch.zeros(grad.shape, dtype=grad.dtype, device=grad.device))
    p.grad = grad
    return p


def test_clip_takes_one_tensor():
    p = param(torch.full((10,), 3.0, device="cuda"))
    assert abs(float(train.clip_grad_norm_(p, 1.0)) - 90.0 ** 0.5) < 1e-5
    assert abs(float(p.grad.norm()) - 1.0) < 1e-5


def test_clip_without_gradients_stays_on_the_device():
    p = torch.nn.Parameter(torch.zeros(4, device="cuda"))
    for arg in (p, [p], []):
        norm = train.clip_grad_norm_(arg, 1.0)
        assert norm.is_cuda and norm.dtype == torch.float32 and norm.shape == (1,) and float(norm) == 0.0
