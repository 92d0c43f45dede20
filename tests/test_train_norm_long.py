"""Layer norm of rows above 8192 columns with many tokens, on side streams and
in graphs.  Bounds as in test_train_norm.py."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

from test_train_norm import EPS, backward, check_backward, check_forward, data, forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,pad,shift", [(300, 8200, 0, 0), (129, 8193, 0, 0), (200, 12288, 8, 0), (257, 16384, 0, 0),
                                           (65, 9001, 3, 1), (64, 8200, 4, 2), (300, 16384, 16, 8)])
def test_long_rows_strided_and_in_place(T, H, pad, shift, dt):
    x, gamma, beta, dy = data(T, H, dt)

    def placed(t):
        buf = torch.full((T * (H + pad) + shift,), 7.0, dtype=dt, device="cuda")
        rows = buf[shift:].as_strided((T, H), (H + pad, 1))
        return buf, rows.copy_(t)

    def between(buf):
        left = torch.ones_like(buf, dtype=torch.bool)
        left[shift:].as_strided((T, H), (H + pad, 1)).fill_(False)
        return bool((buf[left] == 7.0).all())

    (_, xs), (_, ds), (ybuf, ys) = placed(x), placed(dy), placed(torch.zeros_like(x))
    mean, rstd = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    api.moe_nvfp4_layer_norm(xs, gamma, beta, EPS, ys, mean, rstd)
    check_forward(x, gamma, beta, (ys, mean, rstd))
    assert between(ybuf)
    over = xs.clone().as_strided((T, H), (H, 1)) if pad == 0 else placed(x)[1]
    api.moe_nvfp4_layer_norm(over, gamma, beta, EPS, over)
    assert torch.equal(over, ys)
    got = backward(ds, xs, gamma, mean, rstd, dx=ys)
    check_backward(dy, x, gamma, mean, rstd, got)
    assert between(ybuf)
    for which in (ds, xs):
        keep = which.clone()
        again = backward(ds, xs, gamma, mean, rstd, dx=which)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        which.copy_(keep)


@pytest.mark.parametrize("T,H", [(5, 7168), (700, 7168), (700, 1001), (130, 512), (40, 12288)])
def test_on_a_side_stream_and_in_a_graph(T, H):
    x, gamma, beta, dy = data(T, H, torch.bfloat16)
    y, mean, rstd = forward(x, gamma, beta)
    dx, dg, db = backward(dy, x, gamma, mean, rstd)
    keep = (y, mean, rstd, dx, dg, db)
    out = [torch.empty_like(t) for t in keep]
    ws = torch.empty(api.moe_nvfp4_layer_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        api.moe_nvfp4_layer_norm(x, gamma, beta, EPS, out[0], out[1], out[2], side)
        api.moe_nvfp4_layer_norm_backward(dy, x, gamma, out[1], out[2], out[3], out[4], out[5], ws, side)

    torch.cuda.synchronize()
    step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, keep))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, keep))


@pytest.mark.parametrize("sizes", [[700, 5, 100001], [3000] * 200, [5000, 1] * 700])
def test_clipping_in_a_graph(sizes):
    g = torch.Generator("cuda").manual_seed(9)
    t = [torch.randn(n, generator=g, device="cuda").to(torch.bfloat16 if i % 2 else torch.float32)
         for i, n in enumerate(sizes)]
    out = [torch.empty_like(v) for v in t]
    grads = api.GradList(t, out)
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(api.moe_nvfp4_grad_norm_workspace_bytes(len(t)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        api.moe_nvfp4_grad_norm(grads, norm, ws, side)
        api.moe_nvfp4_grad_clip(grads, norm, 0.5, 1e-6, side)

    torch.cuda.synchronize()
    step()
    side.synchronize()
    keep = (norm.clone(), [v.clone() for v in out])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    norm.zero_()
    for v in out:
        v.zero_()
    t[0].mul_(1.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, keep[0]) and all(torch.equal(a, b) for a, b in zip(out, keep[1]))
