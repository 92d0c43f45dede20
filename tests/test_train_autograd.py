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


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_clip_of_gradients_in_other_orders(dt):
    """Transposed and strided gradients (relative bound: a sum of 500 squares and the scaling, three
    roundings of 2^-24 and one of the type)."""
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    wide = r(16, 24)
    grads = [r(12, 20).t(), wide[:, ::2], r(9), r(4, 3, 5).permute(2, 0, 1)]
    rest = wide[:, 1::2].clone()
    want = [v.double() for v in grads]
    total = float(sum(v.square().sum() for v in want).sqrt())
    norm = float(train.clip_grad_norm_([param(v) for v in grads], 1.0))
    assert abs(norm - total) <= 600 * 2.0 ** -24 * total
    half = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    for v, w in zip(grads, want):
        w = w / (norm + 1e-6)
        assert bool(((v.double() - w).abs() <= (half + 4 * 2.0 ** -24) * w.abs() + 1e-38).all())
    assert torch.equal(wide[:, 1::2], rest)


def routes_of(T, E, K, drop, seed=5):
    g = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(T, K, generator=g, device="cuda") < drop] = -1
    return ids, train.sort_routes(ids, E)


def test_row_buffers_smaller_than_the_routes_are_refused():
    ids, routes = routes_of(30, 4, 2, 0.0)
    w = torch.randn(4, 32, 64, device="cuda").bfloat16()
    x = torch.randn(60, 64, device="cuda").bfloat16()
    s = torch.rand(30, 2, device="cuda")
    with pytest.raises(ValueError):
        train.expert_linear(x[:59], w, routes)
    with pytest.raises(ValueError):
        train.combine(x[:59], routes, s)
    # more rows than routes: the rest belongs to no route
    more = torch.cat([x, x[:3]])
    assert torch.equal(train.expert_linear(more, w, routes)[:60], train.expert_linear(x, w, routes))
    assert torch.equal(train.combine(more, routes, s), train.combine(x, routes, s))
