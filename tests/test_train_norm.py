"""Layer norm and its gradient against plain torch in 64 bits.

Bounds, with u = 2^-24 and S = H/32 + 24 (additions in sequence: a row is
spread over 32 threads at least, then a tree):
  mean    d_m = S u mean|x|
  rstd    relative d_r = ((S + 4) u + d_m^2 / var) / 2 + 4 u
  y       |gamma| (|xhat| (d_r + 4 u) + rstd d_m) + 2 u |y| + half an ulp of y
  dx      rstd ((S + 4) u (mean|g| + |xhat| mean|g xhat|) + 8 u (|g| + |mean g| + |xhat mean(g xhat)|)), half an ulp
  dgamma  (T + 8) u sum|dy xhat|,  dbeta (T + 8) u sum|dy|"""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def forward(x, gamma, beta, eps=EPS):
    T, H = x.shape
    y = torch.full((T, H), float("nan"), dtype=x.dtype, device="cuda")
    mean, rstd = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    api.moe_nvfp4_layer_norm(x, gamma, beta, eps, y, mean, rstd)
    return y, mean, rstd


def check_forward(x, gamma, beta, got, eps=EPS):
    H = x.shape[1]
    S = H / 32 + 24
    x64 = x.double()
    m = x64.mean(1)
    var = (x64 - m[:, None]).square().mean(1)
    r = (var + eps).rsqrt()
    y, mean, rstd = got
    dm = S * U * x64.abs().mean(1)
    assert bool(((mean.double() - m).abs() <= dm + U * m.abs()).all())
    dr = ((S + 4) * U + dm.square() / (var + eps)) / 2 + 4 * U
    assert bool(((rstd.double() - r).abs() <= dr * r).all())
    hat = (x64 - m[:, None]) * r[:, None]
    g, b = gamma.double(), 0.0 if beta is None else beta.double()
    want = hat * g + b
    bound = g.abs() * (hat.abs() * (dr + 4 * U)[:, None] + (r * dm)[:, None]) + 2 * U * (want.abs() + (g * hat).abs()) \
        + HALF[x.dtype] * want.abs() * 1.01 + 1e-38
    err = (y.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def backward(dy, x, gamma, mean, rstd, dbeta=True, dx=None):
    T, H = x.shape
    dx = torch.full((T, H), float("nan"), dtype=x.dtype, device="cuda") if dx is None else dx
    dg, db = (torch.full((H,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.full((api.moe_nvfp4_layer_norm_workspace_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    api.moe_nvfp4_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dg, db if dbeta else None, ws)
    return dx, dg, db


def check_backward(dy, x, gamma, mean, rstd, got):
    T, H = x.shape
    S = H / 32 + 24
    dx, dg, db = got
    d, r = dy.double(), rstd.double()[:, None]
    hat = (x.double() - mean.double()[:, None]) * r
    g = d * gamma.double()
    a, b = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
    want = r * (g - a - hat * b)
    bound = r * ((S + 4) * U * (g.abs().mean(1, keepdim=True) + hat.abs() * (g * hat).abs().mean(1, keepdim=True))
                 + 8 * U * (g.abs() + a.abs() + (hat * b).abs())) + HALF[x.dtype] * want.abs() * 1.01 + 1e-38
    err = (dx.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert bool(((dg.double() - (d * hat).sum(0)).abs() <= (T + 8) * U * (d * hat).abs().sum(0) + 1e-38).all())
    assert bool(((db.double() - d.sum(0)).abs() <= (T + 8) * U * d.abs().sum(0) + 1e-38).all())


def data(T, H, dt, seed=0, offset=0.3):
    g = torch.Generator("cuda").manual_seed(seed + 17 * T + H)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = (r(T, H) * (0.5 + torch.rand(H, generator=g, device="cuda")) + offset * r(H)).to(dt)
    return x, 1.0 + 0.2 * r(H), 0.1 * r(H), r(T, H).to(dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7168), (2, 8), (3, 33), (7, 255), (16, 256), (33, 1001), (130, 2048),
                                 (5, 4104), (4, 8192), (3, 16384), (2, 65536), (2, 65535), (1000, 64), (700, 7168),
                                 (1300, 1032), (611, 8192), (2000, 2048), (900, 3001)])
def test_forward_and_backward(T, H, dt):
    x, gamma, beta, dy = data(T, H, dt)
    got = forward(x, gamma, beta)
    check_forward(x, gamma, beta, got)
    check_backward(dy, x, gamma, got[1], got[2], backward(dy, x, gamma, got[1], got[2]))


def test_without_beta_and_statistics():
    x, gamma, beta, dy = data(9, 512, torch.bfloat16)
    y, mean, rstd = forward(x, gamma, None)
    check_forward(x, gamma, None, (y, mean, rstd))
    z = torch.empty_like(y)
    api.moe_nvfp4_layer_norm(x, gamma, None, EPS, z)
    assert torch.equal(y, z)
    a = backward(dy, x, gamma, mean, rstd)
    b = backward(dy, x, gamma, mean, rstd, dbeta=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and bool(torch.isnan(b[2]).all())


def test_a_mean_far_above_the_spread():
    """Rows around 1000 with a spread of 1: the difference of E[x^2] and
    mean^2 would keep no more than four digits in FP32."""
    T, H = 40, 4096
    x, gamma, beta, dy = data(T, H, torch.float32)
    x = x + 1000.0
    check_forward(x, gamma, beta, forward(x, gamma, beta))


def test_constant_rows_and_non_finite_values():
    T, H = 6, 768
    x, gamma, beta, dy = data(T, H, torch.float32)
    x[0] = 0.0
    x[1] = 2.5
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    y, mean, rstd = forward(x, gamma, beta)
    assert torch.allclose(rstd[:2], torch.full((2,), EPS, device="cuda").rsqrt(), rtol=1e-6, atol=0)
    assert torch.equal(y[0], beta)
    assert torch.equal(y[1], beta)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
    check_forward(x[4:], gamma, beta, (y[4:], mean[4:], rstd[4:]))
    # a constant row without eps: 0 * inf
    y, mean, rstd = forward(x[1:2].contiguous(), gamma, beta, 0.0)
    assert bool(torch.isinf(rstd).all()) and bool(torch.isnan(y).all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,pad,shift", [(512, 8, 0), (512, 8, 1), (509, 6, 0), (8, 8, 0)])
def test_strides_shifts_and_in_place(dt, H, pad, shift):
    T = 50
    x, gamma, beta, dy = data(T, H, dt)
    strided = lambda t: torch.zeros(T * (H + pad) + shift, dtype=dt, device="cuda")[shift:].as_strided(
        (T, H), (H + pad, 1)).copy_(t)
    y, mean, rstd = forward(x, gamma, beta)
    xs = strided(x)
    ys = strided(torch.zeros_like(x))
    m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
    api.moe_nvfp4_layer_norm(xs, gamma, beta, EPS, ys, m2, r2)
    check_forward(x, gamma, beta, (ys, m2, r2))
    api.moe_nvfp4_layer_norm(xs, gamma, beta, EPS, xs)
    assert torch.equal(xs, ys)
    dx, dg, db = backward(dy, x, gamma, mean, rstd)
    for over in ("dy", "x"):
        d, v = strided(dy), strided(x)
        got = backward(d, v, gamma, mean, rstd, dx=d if over == "dy" else v)
        check_backward(dy, x, gamma, mean, rstd, got)


# rows that start anywhere within 16 bytes, enough of them for several turns of
# every block; what lies between the rows stays as it is
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,pads,shifts", [
    (613, 513, (0, 0, 0), (0, 0, 0)), (4001, 601, (0, 0, 0), (0, 0, 0)), (7000, 1001, (3, 0, 1), (1, 2, 3)),
    (2500, 1023, (0, 1, 5), (0, 0, 0)), (1300, 1025, (0, 0, 0), (0, 0, 0)), (1300, 1026, (0, 2, 4), (2, 0, 6)),
    (900, 2047, (1, 0, 2), (0, 5, 0)), (700, 4097, (0, 0, 0), (7, 7, 7)), (800, 7167, (0, 0, 0), (0, 0, 0)),
    (650, 8191, (4, 1, 0), (3, 1, 0)), (700, 8190, (0, 0, 0), (0, 0, 0)), (700, 8188, (0, 0, 0), (0, 0, 0)),
    (700, 4096, (1, 8, 0), (0, 0, 1)), (1, 4099, (0, 0, 0), (1, 1, 1)), (160, 1537, (0, 0, 0), (0, 0, 0))])
def test_rows_off_16_byte_blocks(T, H, pads, shifts, dt):
    x, gamma, beta, dy = data(T, H, dt)

    def placed(t, pad, shift):
        buf = torch.full((T * (H + pad) + shift + 16,), 7.0, dtype=dt, device="cuda")
        rows = buf[shift:].as_strided((T, H), (H + pad, 1))
        rows.copy_(t)
        return buf, rows

    def between(buf, pad, shift):
        left = torch.ones_like(buf, dtype=torch.bool)
        left[shift:].as_strided((T, H), (H + pad, 1)).fill_(False)
        return bool((buf[left] == 7.0).all())

    (_, xs), (_, ds), (ybuf, ys) = (placed(t, pads[i], shifts[i]) for i, t in enumerate((x, dy, torch.zeros_like(x))))
    mean, rstd = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    api.moe_nvfp4_layer_norm(xs, gamma, beta, EPS, ys, mean, rstd)
    check_forward(x, gamma, beta, (ys, mean, rstd))
    assert between(ybuf, pads[2], shifts[2])
    got = backward(ds, xs, gamma, mean, rstd, dx=ys)
    check_backward(dy, x, gamma, mean, rstd, got)
    assert between(ybuf, pads[2], shifts[2])
    again = backward(ds, xs, gamma, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for over in (ds, xs):
        keep = over.clone()
        assert torch.equal(backward(ds, xs, gamma, mean, rstd, dx=over)[0], got[0])
        over.copy_(keep)


def test_gradient_against_differences():
    """L = <c, layer_norm(x)> in 64 bits; central differences of step h along v
    are off by O(h^2) of the third derivative."""
    T, H = 5, 96
    x, gamma, beta, c = data(T, H, torch.float32)
    y, mean, rstd = forward(x, gamma, beta)
    dx, dg, db = backward(c, x, gamma, mean, rstd)
    def loss(x, g, b):
        m = x.mean(1, keepdim=True)
        v = (x - m).square().mean(1, keepdim=True)
        return float((((x - m) / (v + EPS).sqrt() * g + b) * c.double()).sum())
    g64 = torch.Generator("cuda").manual_seed(4)
    args = [x.double(), gamma.double(), beta.double()]
    for i, grad in enumerate((dx, dg, db)):
        v = torch.randn(args[i].shape, generator=g64, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        num = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(float((grad.double() * v).sum()) - num) <= 2e-5 * float((grad.double() * v).abs().sum())


def test_no_tokens():
    x, gamma, beta, dy = data(1, 64, torch.bfloat16)
    e = x[:0]
    z = torch.empty(0, device="cuda")
    api.moe_nvfp4_layer_norm(e, gamma, beta, EPS, torch.empty_like(e), z, z.clone())
    dx, dg, db = backward(e, e.clone(), gamma, z, z.clone())
    assert not dg.any() and not db.any()


def test_offsets_beyond_32_bits_and_repeatable():
    T, H = 330000, 7168
    x = torch.randn(T, 64, device="cuda").bfloat16().repeat(1, H // 64)
    _, gamma, beta, _ = data(1, H, torch.bfloat16)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    api.moe_nvfp4_layer_norm(x, gamma, beta, EPS, y, mean, rstd)
    pick = torch.cat([torch.arange(0, 64, device="cuda"), torch.arange(T - 64, T, device="cuda")])
    check_forward(x[pick], gamma, beta, (y[pick], mean[pick], rstd[pick]))
    dx, dg, db = backward(y, x, gamma, mean, rstd)
    d, hat = y[pick].double(), (x[pick].double() - mean[pick].double()[:, None]) * rstd[pick].double()[:, None]
    g = d * gamma.double()
    want = rstd[pick].double()[:, None] * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    assert float((dx[pick].double() - want).norm() / want.norm()) < 2.0 ** -8
    again = backward(y, x, gamma, mean, rstd, dx=dx)
    assert torch.equal(dg, again[1]) and torch.equal(db, again[2])


def test_binding_refuses():
    x, gamma, beta, dy = data(4, 64, torch.bfloat16)
    with pytest.raises(TypeError):
        api.moe_nvfp4_layer_norm(x, gamma.bfloat16(), beta, EPS, torch.empty_like(x))
    with pytest.raises(ValueError):
        api.moe_nvfp4_layer_norm(x, gamma[:32], beta, EPS, torch.empty_like(x))
    with pytest.raises(TypeError):
        api.moe_nvfp4_layer_norm(x, gamma, beta, EPS, torch.empty_like(x, dtype=torch.float32))
    with pytest.raises(api.MoEError):
        api.moe_nvfp4_layer_norm(x, gamma, beta, -1.0, torch.empty_like(x))
