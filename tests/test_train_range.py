"""The range of the gradients' norm, as the header has it: the squares and
their sum are FP32, so a norm above 1.8e19 is infinite, elements below 1e-19
lose digits, and those below 1e-23 add nothing.  Bound: (n / 512 + 100) 2^-24
for the sum, half of it for the root, and where the squares are subnormal
(multiples of 2^-149) half such a multiple for each."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def norm_of(grads):
    norm = torch.full((1,), float("nan"), device="cuda")
    ws = torch.empty(api.moe_nvfp4_grad_norm_workspace_bytes(grads.n), dtype=torch.uint8, device="cuda")
    api.moe_nvfp4_grad_norm(grads, norm, ws)
    return norm


@pytest.mark.parametrize("n,value", [(2, 1.5e19), (1000000, 1e17)])
def test_a_norm_above_the_range_is_infinite(n, value):
    """Every element's square fits, their sum does not; the scale is 0."""
    t = torch.full((n,), value, device="cuda")
    grads = api.GradList([t])
    norm = norm_of(grads)
    assert bool(torch.isinf(norm).all())
    api.moe_nvfp4_grad_clip(grads, norm, 1.0)
    assert not t.any()


@pytest.mark.parametrize("n,value", [(2, 1.2e19), (1000000, 1.7e16), (4, 1e-19), (1000, 1e-21), (7, 1e-22)])
def test_norms_within_the_range(n, value):
    t = torch.full((n,), value, device="cuda")
    square = float(t[0].double()) ** 2
    want = (n * square) ** 0.5
    relative = ((n / 512 + 100) * U + 2.0 ** -150 / square) / 2 + 2 * U
    assert abs(float(norm_of(api.GradList([t])).double()) - want) <= 1.01 * relative * want
