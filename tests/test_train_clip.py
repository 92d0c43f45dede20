"""Global gradient norm and clipping against plain torch in 64 bits.

Bounds, u = 2^-24: a sum of squares of n elements, spread over 512 threads at
least, in any order: relative (n / 512 + 100) u; the root halves it.  The
scaled gradients, given the device's norm: the quotient and the product are
rounded in FP32 (three roundings), then once to the output type."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def norm_of(grads):
    norm = torch.full((1,), float("nan"), device="cuda")
    ws = torch.full((api.moe_nvfp4_grad_norm_workspace_bytes(len(grads.grads)),), 0xFF, dtype=torch.uint8, device="cuda")
    api.moe_nvfp4_grad_norm(grads, norm, ws)
    return norm


def check(tensors, max_norm, out=None, eps=1e-6):
    before = [t.double() for t in tensors]
    grads = api.GradList(tensors, out)
    norm = norm_of(grads)
    total = sum(t.numel() for t in tensors)
    want = float(sum((b.square().sum() for b in before), torch.zeros((), dtype=torch.float64, device="cuda")).sqrt())
    assert abs(float(norm) - want) <= ((total / 512 + 100) * U / 2 + 2 * U) * want
    api.moe_nvfp4_grad_clip(grads, norm, max_norm, eps)
    scale = min(1.0, max_norm / (float(norm) + eps))
    for b, o in zip(before, grads.out):
        err = (o.double() - b * scale).abs()
        assert bool((err <= (HALF[o.dtype] + 4 * U) * (b * scale).abs() + 1e-38).all())
    return norm


def normal(sizes, dts, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(n, generator=g, device="cuda").mul_(0.5 + i % 3).to(dts[i % len(dts)]) for i, n in enumerate(sizes)]


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16385], [3, 1, 2], [100003, 8, 1, 65536], [33] * 95, [33] * 97,
                                   [1000] * 300, [0, 5, 0, 9, 0], [2000000, 5, 3000001]])
@pytest.mark.parametrize("dts", [[BF], [F32], [BF, F32]])
@pytest.mark.parametrize("max_norm", [0.7, 1e9])
def test_norm_and_clip(sizes, dts, max_norm):
    tensors = normal(sizes, dts)
    check(tensors, max_norm, [torch.full_like(t, float("nan")) for t in tensors])
    check(tensors, max_norm)                               # in place


# lists that take one round of the blocks and several, every size of the
# argument, and more tensors than one launch holds; empty tensors between
@pytest.mark.parametrize("sizes", [[20001, 1, 0] * 80, [40000] * 400, [5000, 1, 30000] * 400, [4096] * 608, [4097] * 609,
                                   [0] * 1000 + [77, 0, 200000], [17, 3000000, 9] * 12, [250001] * 33, [1] * 1921])
@pytest.mark.parametrize("dts", [[BF], [F32, BF, BF]])
def test_many_tensors(sizes, dts):
    tensors = normal(sizes, dts, seed=1)
    first = check(tensors, 0.5, [torch.full_like(t, float("nan")) for t in tensors])
    again = norm_of(api.GradList(tensors, None))
    assert torch.equal(first, again)


def test_shifted_pointers():
    base = normal([40000], [BF])[0]
    tensors = [base[1:20000], base[20001:20009], base[20010:39999]]
    out = torch.zeros_like(base)
    check(tensors, 0.5, [out[1:20000], out[20001:20009], out[20010:39999]])
    assert not out[:1].any() and not out[20000:20001].any() and not out[20009:20010].any() and not out[39999:].any()
    # input aligned, output not
    check([base[:1000]], 0.5, [out[3:1003]])


def test_no_gradients():
    norm = norm_of(api.GradList([]))
    assert float(norm) == 0.0
    api.moe_nvfp4_grad_clip(api.GradList([]), norm, 1.0)
    norm = norm_of(api.GradList([torch.empty(0, device="cuda")]))
    assert float(norm) == 0.0


def test_zero_and_non_finite_gradients():
    z = [torch.zeros(1000, device="cuda")]
    assert float(check(z, 1.0)) == 0.0
    for bad in (float("inf"), float("nan")):
        t = normal([5000], [F32])
        t[0][17] = bad
        grads = api.GradList(t, [torch.empty_like(t[0])])
        norm = norm_of(grads)
        assert (torch.isinf if bad == float("inf") else torch.isnan)(norm).all()
        api.moe_nvfp4_grad_clip(grads, norm, 1.0)
        out = grads.out[0]
        if bad == float("inf"):      # scale 0: zeros, and NaN where the infinity was
            assert torch.isnan(out[17]) and int((out == 0).sum()) == 4999
        else:
            assert bool(torch.isnan(out).all())


def test_range_of_the_squares():
    """Documented: beyond 1.8e19 the squares overflow, below 1e-23 they vanish."""
    assert torch.isinf(norm_of(api.GradList([torch.full((4,), 3e19, device="cuda")]))).all()
    assert float(norm_of(api.GradList([torch.full((4,), 1e-24, device="cuda")]))) == 0.0
    n = norm_of(api.GradList([torch.full((4,), 1e18, device="cuda")]))
    assert abs(float(n) - 2e18) <= 1e-6 * 2e18


def test_unclipped_in_place_keeps_bits():
    t = normal([70000, 11], [BF])
    keep = [v.clone() for v in t]
    grads = api.GradList(t)
    api.moe_nvfp4_grad_clip(grads, norm_of(grads), 1e6)
    assert all(torch.equal(a, b) for a, b in zip(t, keep))


def test_repeatable_and_on_a_side_stream():
    t = normal([3000000, 17, 400000], [BF, F32])
    grads = api.GradList(t, [torch.empty_like(v) for v in t])
    a, b = norm_of(grads), norm_of(grads)
    assert torch.equal(a, b)
    side = torch.cuda.Stream()
    ws = torch.empty(api.moe_nvfp4_grad_norm_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    c = torch.empty_like(a)
    torch.cuda.synchronize()
    api.moe_nvfp4_grad_norm(grads, c, ws, side)
    api.moe_nvfp4_grad_clip(grads, c, 1.0, 1e-6, side)
    side.synchronize()
    assert torch.equal(a, c)
    got = [o.clone() for o in grads.out]
    api.moe_nvfp4_grad_clip(grads, a, 1.0, 1e-6)
    assert all(torch.equal(x, y) for x, y in zip(got, grads.out))


def test_more_than_2_31_elements():
    n = 2 ** 31 + 4099
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[:3], t[-5:] = 2.0, 1.0
    grads = api.GradList([t])
    norm = norm_of(grads)
    assert abs(float(norm) - 17.0 ** 0.5) <= 4 * U * 17.0 ** 0.5
    api.moe_nvfp4_grad_clip(grads, norm, 17.0 ** 0.5 / 2, 0.0)
    assert bool((t[:3] == 1.0).all()) and bool((t[-5:] == 0.5).all()) and int((t != 0).sum()) == 8


def test_binding_refuses():
    g = torch.zeros(8, device="cuda")
    with pytest.raises(TypeError):
        api.GradList([g.half()])
    with pytest.raises(TypeError):
        api.GradList([g], [g.bfloat16()])
    with pytest.raises(ValueError):
        api.GradList([g], [g[:4]])
    with pytest.raises(ValueError):
        api.GradList([torch.zeros(8, 8, device="cuda").t()])
    with pytest.raises(api.MoEError):
        api.moe_nvfp4_grad_clip(api.GradList([g]), torch.zeros(1, device="cuda"), -1.0)
