"""train.py beside the block: what its functions do with dropped routes, row
buffers of another size, odd gradients, and errors found on the device."""
import threading
import time

import pytest
import torch
import torch.nn.functional as F

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


def test_a_list_of_another_device_than_the_norm_is_refused():
    """The list's device is claimed, not real: its tensors stay where they are."""
    g, norm, ws = torch.ones(8, device="cuda"), torch.full((1,), 7.0, device="cuda"), torch.zeros(256 * 1024, device="cuda")
    grads = api.GradList([g])
    assert grads.index == 0
    grads.index = 1
    with pytest.raises(ValueError, match="device"):
        api.moe_nvfp4_grad_norm(grads, norm, ws)
    with pytest.raises(ValueError, match="device"):
        api.moe_nvfp4_grad_clip(grads, norm, 1.0)
    torch.cuda.synchronize()
    assert float(norm) == 7.0 and bool((g == 1.0).all())


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


@pytest.mark.parametrize("T,drop", [(40, 0.3), (300, 0.9), (7, 1.0), (64, 0.0)])
def test_parameters_between_products_with_dropped_routes(monkeypatch, T, drop):
    """A scale and a bias per channel between two products, every buffer full
    of NaN before it is written: the rows that no route owns are zeros and add
    nothing to their gradients.  Bound: z, the activation, do and da are
    rounded to BF16 once each (half an ulp is 2^-8), the rest is FP32."""
    empty, empty_like = torch.empty, torch.empty_like
    spoil = lambda t: t.fill_(float("nan")) if t.is_floating_point() else t
    monkeypatch.setattr(torch, "empty", lambda *a, **k: spoil(empty(*a, **k)))
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: spoil(empty_like(*a, **k)))
    H, N, E, K = 64, 96, 5, 3
    ids, routes = routes_of(T, E, K, drop)
    g = torch.Generator("cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = r(T, H).bfloat16().requires_grad_(True)
    w1 = (r(E, N, H) * H ** -0.5).bfloat16().requires_grad_(True)
    w2 = (r(E, H, N) * N ** -0.5).bfloat16().requires_grad_(True)
    scale, bias = (1.0 + 0.2 * r(N)).requires_grad_(True), (0.1 * r(N)).requires_grad_(True)
    s = torch.rand(T, K, generator=g, device="cuda").requires_grad_(True)
    z = train.expert_linear(train.dispatch(x, routes), w1, routes)
    z.retain_grad()
    a = F.silu(z.float() * scale + bias).bfloat16()
    a.retain_grad()
    o = train.expert_linear(a, w2, routes)
    y = train.combine(o, routes, s)
    c = r(T, H).bfloat16()
    y.backward(c)
    used = int(routes.used)
    for t in (z, o, a.grad):
        assert not t[used:].any()
    x2, w1_2, w2_2, sc2, b2, s2 = (v.detach().double().requires_grad_(True) for v in (x, w1, w2, scale, bias, s))
    e = ids.clamp(min=0).long()
    z2 = torch.einsum("th,tknh->tkn", x2, w1_2[e])
    o2 = torch.einsum("tkn,tkhn->tkh", F.silu(z2 * sc2 + b2), w2_2[e])
    (o2 * torch.where(ids >= 0, s2, 0.0)[..., None]).sum(1).backward(c.double())
    for got, want in ((x, x2), (w1, w1_2), (w2, w2_2), (scale, sc2), (bias, b2), (s, s2)):
        err = float((got.grad.double() - want.grad).norm())
        assert err <= 5 * 2.0 ** -8 * float(want.grad.norm()), err


@pytest.mark.parametrize("rows,used,H,dt", [(1, 0, 8, torch.bfloat16), (31, 4, 33, torch.float32), (5000, 3, 72, torch.bfloat16),
                                            (4097, 4096, 1001, torch.bfloat16), (70001, 11, 260, torch.float32),
                                            (2100, -5, 7168, torch.bfloat16), (40, 40, 64, torch.float32)])
def test_a_dispatch_of_no_tokens_clears_rows(rows, used, H, dt):
    out = torch.full((rows, H), 7.0, dtype=dt, device="cuda")
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    api.moe_nvfp4_dispatch(out[:0], none, torch.tensor([used], dtype=torch.int32, device="cuda"), out)
    keep = max(used, 0)
    assert bool((out[:keep] == 7.0).all()) and not out[keep:].any()
    out.fill_(7.0)
    api.moe_nvfp4_dispatch(None, None, torch.tensor([used], dtype=torch.int32, device="cuda"), out)
    assert bool((out[:keep] == 7.0).all()) and not out[keep:].any()
    with pytest.raises(TypeError):
        api.moe_nvfp4_dispatch(None, none, None, out)
    with pytest.raises(TypeError):
        api.moe_nvfp4_dispatch(out[:0], None, None, out)


def test_bad_segments_are_reported():
    ids, routes = routes_of(30, 4, 2, 0.0)
    x = torch.randn(60, 64, device="cuda").bfloat16().requires_grad_(True)
    w = torch.randn(4, 32, 64, device="cuda").bfloat16().requires_grad_(True)
    y = train.expert_linear(x, w, routes)
    routes.check()
    keep = routes.count.clone()
    routes.count[3] += 1000                     # past the buffer's end
    for call in (lambda: train.expert_linear(x, w, routes),
                 lambda: torch.autograd.grad(y, x, torch.ones_like(y), retain_graph=True),
                 lambda: torch.autograd.grad(y, w, torch.ones_like(y), retain_graph=True)):
        call()
        with pytest.raises(api.MoEError) as err:
            routes.check()
        assert err.value.code == api.MOE_ERR_INVALID_ARG
        routes.check()                          # reported once
    routes.count.copy_(keep)
    y.sum().backward()
    routes.check()


def test_other_threads_run_while_a_launch_waits():
    """A launch into a full queue waits for the device; the interpreter is free
    meanwhile.  The queue fills behind a kernel of half a second and more."""
    x, gamma = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    y, side = torch.empty_like(x), torch.cuda.Stream()
    api.moe_nvfp4_layer_norm(x, gamma, None, 1e-5, y)
    torch.cuda.synchronize()
    took = []

    def work():
        t0 = time.perf_counter()
        for _ in range(6000):
            api.moe_nvfp4_layer_norm(x, gamma, None, 1e-5, y, None, None, side)
        took.append(time.perf_counter() - t0)

    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000_000)
    worker = threading.Thread(target=work)
    longest, last = 0.0, time.perf_counter()
    worker.start()             # may come back only once the worker's launch does
    while worker.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        longest, last = max(longest, now - last), now
    worker.join()
    torch.cuda.synchronize()
    assert took[0] > 0.3, "the queue never filled"
    assert longest < 0.5 * took[0], (longest, took[0])


def test_transforms_without_a_rule_raise():
    gamma = torch.ones(64, device="cuda")
    x = torch.randn(3, 5, 64, device="cuda")
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda v: train.layer_norm(v, gamma))(x)
    with pytest.raises((RuntimeError, NotImplementedError)):
        torch.func.jvp(lambda v: train.layer_norm(v, gamma), (x[0],), (x[1],))
    v = x[1].clone().requires_grad_(True)
    (d,) = torch.autograd.grad(train.layer_norm(v, gamma).square().sum(), v, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()


def test_routes_of_host_tensors_are_a_type_error():
    with pytest.raises(TypeError):
        train.sort_routes(torch.zeros(4, 2, dtype=torch.int32), 8)


def test_routes_first_sorted_in_a_graph(monkeypatch):
    """The status word is then the graph's own, cleared by its replays."""
    monkeypatch.setattr(train, "_status_words", {})
    ids, _ = routes_of(30, 4, 2, 0.0)
    monkeypatch.setattr(train, "_status_words", {})
    x, w = torch.randn(60, 64, device="cuda").bfloat16(), torch.randn(4, 32, 64, device="cuda").bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        routes = train.sort_routes(ids, 4)
        y = train.expert_linear(x, w, routes)
    graph.replay()
    routes.check()
    again = train.sort_routes(ids, 4)
    assert again.status.data_ptr() != routes.status.data_ptr()
    assert torch.equal(train.expert_linear(x, w, again), y)
    again.check()
