"""RMS norm with the residual's addition, and its gradient, against plain torch in
64 bits.

Bounds, with u = 2^-24 and S = H/32 + 24 (additions in sequence: a row is spread
over 32 threads at least, then a tree):
  h       equal to torch's sum, rounded once
  rstd    relative d_r = (S + 4) u / 2 + 4 u
  y       (d_r + 4 u) |y| and half a unit of its type
  scales  relative d_r + 6 u; powers of two equal but where the block's largest |y|
          is within that of a power of two
  q       by the kernel's own scale: half a step of E4M3 (2^-4 of the value, 2^-10
          of the scale at least), what lies above 448, and y's (d_r + 8 u)
  dx      rstd ((S + 8) u |hhat| mean|g hhat| + 8 u (|g| + |hhat mean(g hhat)|)) + 4 u |dh|, half a unit
  dgamma  (T + 8) u sum|dy hhat|"""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build, train

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
NAN = float("nan")
MODES = [None, "row", "block", "mx"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def inputs(T, H, dt, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed * 7919 + T * 31 + H)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
    x = (scale * r(T, H) * (0.5 + torch.rand(H, generator=g, device="cuda"))).to(dt)
    return x, (2 * scale * r(T, H)).to(dt), 1.0 + 0.2 * r(H)


def scales_for(mode, T, H):
    if mode == "row":
        return torch.full((T,), NAN, device="cuda")
    if mode == "block":
        return torch.full((T, -(-H // 128)), NAN, device="cuda")
    return torch.full((T, -(-H // 32)), 0xEE, dtype=torch.uint8, device="cuda")


def forward(x, res, gamma, mode=None, eps=EPS, h=None, y=None, with_y=True, stream=None):
    """(h, y, q, scales, rstd)."""
    T, H = x.shape
    new = lambda: torch.full((T, H), NAN, dtype=x.dtype, device="cuda")      # noqa: E731
    h = (new() if h is None else h) if res is not None else None
    y = (new() if y is None else y) if with_y else None
    q = scales = None
    if mode is not None:
        q, scales = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), scales_for(mode, T, H)
    rstd = torch.full((T,), NAN, device="cuda")
    api.moe_nvfp4_rms_norm(x, res, gamma, eps, h, y, q, scales, rstd, stream)
    return h, y, q, scales, rstd


def check_forward(x, res, gamma, got, mode=None, eps=EPS):
    T, H = x.shape
    h, y, q, scales, rstd = got
    s = x
    if res is not None:
        s = (x.float() + res.float()).to(x.dtype)
        assert torch.equal(h, s)
    s = s.double()
    r = (s.square().mean(1) + eps).rsqrt()
    dr = (H / 32 + 28) * U / 2 + 4 * U
    assert bool(((rstd.double() - r).abs() <= dr * r).all())
    want = s * r[:, None] * gamma.double()
    if y is not None:
        err = (y.double() - want).abs()
        bound = (dr + 4 * U + 1.01 * HALF[x.dtype]) * want.abs() + 1e-38
        assert bool((err <= bound).all()), float((err / bound).max())
    if mode is None:
        return
    n = {"row": H, "block": 128, "mx": 32}[mode]
    pad = torch.nn.functional.pad(want, (0, -H % n)).view(T, -1, n)
    most = pad.abs().amax(2)
    if mode == "mx":
        got_s = torch.ldexp(torch.ones_like(most), scales.double().int() - 127)
        lo, hi = (torch.frexp(most * (1 + f * (dr + 6 * U))).exponent - 9 for f in (-1, 1))
        e = scales.int() - 127
        zero = most == 0
        assert bool(((e >= lo.clamp(-127, 127)) & (e <= hi.clamp(-127, 127)) | zero).all()) and bool((e[zero] == -127).all())
    else:
        got_s = scales.view(T, -1).double()
        true = torch.where(most > 0, (most / 448).clamp(min=2.0 ** -126), 1.0)
        assert bool(((got_s - true).abs() <= (dr + 6 * U) * true).all())
    value = torch.nn.functional.pad(q.float(), (0, -H % n)).double().view(T, -1, n) * got_s[:, :, None]
    over = (pad.abs() - 448 * got_s[:, :, None]).clamp(min=0)
    bound = torch.maximum(pad.abs() * 2.0 ** -4, got_s[:, :, None] * 2.0 ** -10) * 1.001 + over + (dr + 8 * U) * pad.abs()
    err = (value - pad).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())


SHAPES = [(1, 1), (3, 7), (2, 31), (5, 32), (1, 64), (40, 33), (7, 100), (9, 128), (33, 129), (160, 136), (3, 250), (700, 256), (4, 510),
          (17, 1000), (1023, 1001), (5, 1024), (300, 1032), (2, 2050), (31, 2047), (6, 4096), (1, 7168), (613, 7168), (2, 7167),
          (5, 8192), (3, 8200), (2, 8193), (4, 16384), (1, 65536), (2, 65535)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mode", MODES)
def test_forward(T, H, dt, mode):
    x, res, gamma = inputs(T, H, dt)
    check_forward(x, None, gamma, forward(x, None, gamma, mode), mode)
    got = forward(x, res, gamma, mode)
    check_forward(x, res, gamma, got, mode)
    if mode is not None:        # without y, and without h
        again = forward(x, res, gamma, mode, with_y=False)
        assert torch.equal(again[2].view(torch.uint8), got[2].view(torch.uint8)) and torch.equal(again[3], got[3])
        q, s = torch.empty_like(got[2]), torch.empty_like(got[3])
        api.moe_nvfp4_rms_norm(x, res, gamma, EPS, None, None, q, s)
        assert torch.equal(q.view(torch.uint8), got[2].view(torch.uint8)) and torch.equal(s, got[3])


@pytest.mark.parametrize("H", [64, 1000, 1001, 7168, 9000])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mode", [None, "mx"])
def test_in_place(H, dt, mode):
    x, res, gamma = inputs(37, H, dt)
    want = forward(x, res, gamma, mode)
    plain = forward(x, None, gamma, mode)
    same = lambda a, b: all(u is None or torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))   # noqa: E731
    for take in ("h=res", "h=x", "y=x,h=res", "y=res,h=x", "y=x"):
        a, r = x.clone(), res.clone()
        if take == "y=x":
            assert same(forward(a, None, gamma, mode, y=a), plain)
        else:
            h = r if "h=res" in take else a
            y = a if "y=x" in take else r if "y=res" in take else None
            assert same(forward(a, r, gamma, mode, h=h, y=y), want)


@pytest.mark.parametrize("H", [64, 100, 1001, 7168])
@pytest.mark.parametrize("dt", [BF, F32])
def test_strided(H, dt):
    """Columns of wider tensors, at odd offsets too; what lies around them stays."""
    x, res, gamma = inputs(45, H, dt)
    want = forward(x, res, gamma, "row")
    for wide, at in ((H + 16, 8), (H + 5, 3), (3 * H, H)):
        buf = [torch.full((45, wide), 7.0, dtype=dt, device="cuda") for _ in range(4)]
        v = [b[:, at:at + H] for b in buf]
        v[0].copy_(x)
        v[1].copy_(res)
        got = forward(v[0], v[1], gamma, "row", h=v[2], y=v[3])
        check_forward(x, res, gamma, (got[0].contiguous(), *got[1:]), "row")
        assert torch.equal(got[0], want[0])
        for b in buf:
            b[:, at:at + H] = 7.0
            assert bool((b == 7.0).all())


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("H", [40, 1000, 9000])
def test_zero_and_not_finite_rows(mode, H):
    x, _, gamma = inputs(6, H, F32)
    x[1] = 0.0
    x[2, 5] = NAN
    x[3, 7] = float("inf")
    x[4] *= 1e-30
    h, y, q, s, rstd = forward(x, None, gamma, mode)
    keep = [0, 1, 4, 5]
    check_forward(x[keep].contiguous(), None, gamma, (None, y[keep].contiguous(), None if q is None else q[keep].contiguous(),
                                                      None if s is None else s[keep].contiguous(), rstd[keep].contiguous()), mode)
    assert not y[1].any() and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3, 7]))
    if q is not None:
        assert bool((q[1].float() == 0).all()) and bool(torch.isnan(q[2].float()).all()) and bool(torch.isnan(q[3, 7].float()))
        s = s.view(6, -1)
        assert bool((s[1] == (0 if mode == "mx" else 1)).all())


def test_small_results_keep_a_finite_scale():
    x, _, gamma = inputs(3, 256, F32)
    for tiny in (1e-36, 1e-39, 0.0):
        for mode in ("row", "block", "mx"):
            got = forward(x, None, gamma * tiny, mode)
            assert bool(torch.isfinite(got[2].float()).all())
            if tiny == 1e-36:
                check_forward(x, None, gamma * tiny, got, mode)


def backward(dy, dh, h, gamma, rstd, dx=None):
    T, H = h.shape
    dx = torch.full((T, H), NAN, dtype=h.dtype, device="cuda") if dx is None else dx
    dg = torch.full((H,), NAN, device="cuda")
    ws = torch.full((api.moe_nvfp4_rms_norm_workspace_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    api.moe_nvfp4_rms_norm_backward(dy, dh, h, gamma, rstd, dx, dg, ws)
    return dx, dg


def check_backward(dy, dh, h, gamma, rstd, got):
    T, H = h.shape
    S = H / 32 + 24
    dx, dg = got
    d, hat, r = dy.double(), h.double() * rstd.double()[:, None], rstd.double()[:, None]
    g = d * gamma.double()
    mean, amean = (g * hat).mean(1, keepdim=True), (g * hat).abs().mean(1, keepdim=True)
    want = r * (g - hat * mean)
    bound = r * ((S + 8) * U * hat.abs() * amean + 8 * U * (g.abs() + (hat * mean).abs()))
    if dh is not None:
        want = want + dh.double()
        bound = bound + 4 * U * dh.double().abs()
    bound = bound + 1.01 * HALF[h.dtype] * want.abs() + 1e-38
    err = (dx.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    err, bound = (dg.double() - (d * hat).sum(0)).abs(), (T + 8) * U * (d * hat).abs().sum(0) + 1e-38
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("T,H", SHAPES + [(2000, 64), (1300, 72), (5000, 1000), (1217, 1040), (900, 3000), (700, 8192), (650, 7167),
                                          (2500, 250), (153, 4104), (400, 8200)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward(T, H, dt, with_dh):
    x, res, gamma = inputs(T, H, dt)
    dy, dh, _ = inputs(T, H, dt, seed=1)
    dh = dh if with_dh else None
    rstd = (x.double().square().mean(1) + EPS).rsqrt().float()
    got = backward(dy, dh, x, gamma, rstd)
    check_backward(dy, dh, x, gamma, rstd, got)
    again = backward(dy, dh, x, gamma, rstd)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("T,H", [(37, 64), (37, 1001), (700, 1024), (400, 7168), (33, 9000), (313, 1032)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_backward_in_place_and_strided(T, H, dt):
    x, _, gamma = inputs(T, H, dt)
    dy, dh, _ = inputs(T, H, dt, seed=1)
    rstd = (x.double().square().mean(1) + EPS).rsqrt().float()
    want = backward(dy, dh, x, gamma, rstd)
    for which in range(3):
        v = [dy.clone(), dh.clone(), x.clone()]
        got = backward(v[0], v[1], v[2], gamma, rstd, dx=v[which])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for wide, at in ((H + 16, 8), (H + 5, 3)):
        buf = [torch.full((T, wide), 7.0, dtype=dt, device="cuda") for _ in range(4)]
        v = [b[:, at:at + H] for b in buf]
        for a, b in zip(v, (dy, dh, x)):
            a.copy_(b)
        got = backward(v[0], v[1], v[2], gamma, rstd, dx=v[3])
        check_backward(dy, dh, x, gamma, rstd, (got[0].contiguous(), got[1]))
        for b in buf:
            b[:, at:at + H] = 7.0
            assert bool((b == 7.0).all())


@pytest.mark.parametrize("T,H", [(153, 8256), (200, 16384), (160, 12296), (154, 16392)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mode", MODES)
def test_forward_of_many_long_rows(T, H, dt, mode):
    x, res, gamma = inputs(T, H, dt)
    check_forward(x, res, gamma, forward(x, res, gamma, mode), mode)


@pytest.mark.parametrize("T,H", [(200, 16384), (1000, 9000), (321, 12300), (130, 16392), (257, 9001), (65, 40000)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward_of_many_long_rows(T, H, dt, with_dh):
    test_backward(T, H, dt, with_dh)


@pytest.mark.parametrize("T,H", [(2600, 1001), (400, 7167), (200, 16384)])
def test_backward_in_place_of_rows_under_way(T, H):
    """A block copies its next row while dx goes over an earlier one."""
    test_backward_in_place_and_strided(T, H, BF)


def test_backward_against_differences():
    """Central differences of sum(dy y) in 64 bits, h = 1e-5: off by h^2 and 1e-16 / h, on gradients of up to
    10; the kernel's own error is below 1e-5 (H = 24: 50 units of 2^-24)."""
    T, H, step = 3, 24, 1e-5
    x, res, gamma = inputs(T, H, F32)
    dy, dh, _ = inputs(T, H, F32, seed=1)
    h, y, _, _, rstd = forward(x, res, gamma)
    dx, dg = backward(dy, dh, h, gamma, rstd)
    f = lambda h, g: ((h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * g) * dy.double()).sum(1) + (h * dh.double()).sum(1)  # noqa: E731
    h64, g64 = h.double(), gamma.double()
    for i in range(H):
        e = torch.zeros(H, dtype=torch.float64, device="cuda")
        e[i] = step
        d = (f(h64 + e, g64) - f(h64 - e, g64)) / (2 * step)
        assert bool(((dx[:, i] - d).abs() <= 2e-5).all())
        d = (f(h64, g64 + e) - f(h64, g64 - e)).sum() / (2 * step)
        assert abs(float(dg[i]) - float(d)) <= 2e-5


def test_empty():
    gamma = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    api.moe_nvfp4_rms_norm(x, None, gamma, EPS, None, torch.empty_like(x))
    _, dg = backward(x, None, x, gamma, torch.empty(0, device="cuda"))
    assert not dg.any()


@pytest.mark.parametrize("dt", [BF, F32])
def test_autograd(dt):
    """Against autograd in 64 bits on the same h: the dx bound above, with dy and dh of the output's gradients."""
    x, res, gamma = inputs(70, 264, dt)
    dy, dh, _ = inputs(70, 264, dt, seed=2)
    xl, rl, gl = x.clone().requires_grad_(True), res.clone().requires_grad_(True), gamma.clone().requires_grad_(True)
    y, h = train.rms_norm(xl, gl, rl)
    (y.float() * dy.float()).sum().add((h.float() * dh.float()).sum()).backward()
    rstd = (h.detach().double().square().mean(1) + EPS).rsqrt().float()
    check_backward(dy, dh, h.detach(), gamma, rstd, (xl.grad, gl.grad))
    assert torch.equal(xl.grad, rl.grad) and xl.grad.data_ptr() != rl.grad.data_ptr()
    # only h used, only y used, no residual
    xl.grad = rl.grad = gl.grad = None
    _, h = train.rms_norm(xl, gl, rl)
    h.backward(dh)
    assert torch.equal(xl.grad, dh) and torch.equal(rl.grad, dh) and gl.grad is None
    xl.grad = None
    train.rms_norm(xl, gl).backward(dy)
    rstd = (x.double().square().mean(1) + EPS).rsqrt().float()
    check_backward(dy, None, x, gamma, rstd, (xl.grad, gl.grad))


@pytest.mark.parametrize("T,H", [(50, 512), (700, 7168), (613, 1001), (5, 9000)])
def test_streams_and_graphs(T, H):
    x, res, gamma = inputs(T, H, BF)
    dy, dh, _ = inputs(T, H, BF, seed=1)
    want = forward(x, res, gamma, "mx")
    back = backward(dy, dh, want[0], gamma, want[4])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = forward(x, res, gamma, "mx", stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    static = [v.clone() for v in (x, res, dy, dh)]
    out = [torch.empty_like(v) for v in (x, x, x)]
    q, s, rstd, dg = torch.empty_like(want[2]), torch.empty_like(want[3]), torch.empty_like(want[4]), torch.empty(H, device="cuda")
    ws = torch.empty(api.moe_nvfp4_rms_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_nvfp4_rms_norm(static[0], static[1], gamma, EPS, out[0], out[1], q, s, rstd)
        api.moe_nvfp4_rms_norm_backward(static[2], static[3], out[0], gamma, rstd, out[2], dg, ws)
    for _ in range(2):
        for o in out:
            o.fill_(NAN)
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(s, want[3])
        assert torch.equal(q.view(torch.uint8), want[2].view(torch.uint8))
        assert torch.equal(out[2], back[0]) and torch.equal(dg, back[1])
    x2, _, _ = inputs(T, H, BF, seed=5)
    static[0].copy_(x2)
    graph.replay()
    assert torch.equal(out[1], forward(x2, res, gamma)[1])


def test_binding_refuses():
    x, res, gamma = inputs(4, 64, BF)
    q, s = torch.empty(4, 64, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, device="cuda")
    y = torch.empty_like(x)
    f = lambda x=x, res=None, gamma=gamma, h=None, y=y, q=None, s=None, r=None: api.moe_nvfp4_rms_norm(x, res, gamma, EPS, h, y, q, s, r)  # noqa: E731
    for kw in (dict(x=x.half()), dict(x=x.cpu()), dict(y=y.float()), dict(res=res.float()), dict(gamma=gamma.bfloat16()),
               dict(q=q.view(torch.uint8), s=s), dict(q=q, s=s.double()), dict(q=q, s=s.view(torch.int32)), dict(r=s.double())):
        with pytest.raises(TypeError):
            f(**kw)
    for kw in (dict(res=res[:3]), dict(y=y[:, :32]), dict(gamma=gamma[:32]), dict(q=q), dict(s=s), dict(q=q[:, :32], s=s),
               dict(q=q, s=s[:3]), dict(q=q, s=s[:, None].repeat(1, 2)), dict(r=s[:2]), dict(q=q.t(), s=s),
               dict(q=q, s=torch.empty(4, 3, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            f(**kw)
    for kw in (dict(y=None), dict(h=torch.empty_like(x)), dict(res=res, h=y, y=y)):
        with pytest.raises(api.MoEError):
            f(**kw)
