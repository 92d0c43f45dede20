"""Layer norm between columns of one buffer.  Bounds as in test_train_norm.py."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

from test_train_norm import EPS, backward, check_backward, check_forward, data

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,first,second", [(700, 2048, 0, 2048), (700, 1001, 1003, 0), (33, 256, 264, 0),
                                              (9, 8200, 0, 8200), (1300, 513, 0, 513)])
def test_disjoint_columns_of_one_buffer(T, H, first, second, dt):
    """Rows of input and output side by side in one buffer share no element."""
    x, gamma, beta, dy = data(T, H, dt)
    buf = torch.full((T, max(first, second) + H + 3), 7.0, dtype=dt, device="cuda")
    xs, ys = buf[:, first:first + H], buf[:, second:second + H]
    xs.copy_(x)
    left = torch.ones_like(buf, dtype=torch.bool)
    left[:, second:second + H] = False
    keep = buf.clone()
    mean, rstd = (torch.empty(T, device="cuda") for _ in range(2))
    api.moe_nvfp4_layer_norm(xs, gamma, beta, EPS, ys, mean, rstd)
    check_forward(x, gamma, beta, (ys, mean, rstd))
    check_backward(dy, x, gamma, mean, rstd, backward(dy, xs, gamma, mean, rstd, dx=ys))
    assert torch.equal(buf[left], keep[left])
