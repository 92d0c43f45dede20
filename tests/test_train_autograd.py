"""train.py beside the block: what its functions do with dropped routes, row
buffers of another size, odd gradients, and errors found on the device."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

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
