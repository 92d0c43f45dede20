"""The experts' products and their gradients against plain torch in 64 bits.

Bound: BF16 products are exact in FP32; a sum of D of them in any order has at
most D + 4 roundings of 2^-24 of the sum of the absolute products, then half an
ulp (2^-8: eight significant bits) of the BF16 result."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def segments(counts, gaps=0):
    """count and offsets of segments in order, `gaps` rows of no expert before each; rows in all."""
    off, at = [], 0
    for c in counts:
        at += gaps
        off.append(at)
        at += c
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(counts, **i32), torch.tensor(off, **i32), at + gaps


def check(got, want, mag, D, what):
    err = (got.double() - want).abs()
    bound = 2.0 ** -8 * want.abs() * 1.01 + (D + 4) * U * mag + 1e-38
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


def run_all(counts, N, K, gaps=0, seed=0, poison=True, status=None, streams=None):
    g = torch.Generator("cuda").manual_seed(seed + N + K + sum(counts))
    count, offsets, R = segments(counts, gaps)
    E = len(counts)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    x, dy = r(R, K), r(R, N)
    w = (r(E, N, K) * K ** -0.5).bfloat16()
    owned = torch.zeros(R, dtype=torch.bool, device="cuda")
    for c, o in zip(counts, offsets.tolist()):
        owned[o:o + c] = True
    if poison:
        x[~owned] = float("nan")
        dy[~owned] = float("inf")
    y = torch.full((R, N), 9.0, dtype=x.dtype, device="cuda")
    dx = torch.full((R, K), 9.0, dtype=x.dtype, device="cuda")
    dw = torch.full((E, N, K), float("nan"), dtype=x.dtype, device="cuda")
    api.moe_nvfp4_expert_linear(x, w, count, offsets, y, status)
    api.moe_nvfp4_expert_linear_dgrad(dy, w, count, offsets, dx, status)
    api.moe_nvfp4_expert_linear_wgrad(dy, x, count, offsets, dw, status)
    assert bool((y[~owned] == 9.0).all()) and bool((dx[~owned] == 9.0).all())
    for e, (c, o) in enumerate(zip(counts, offsets.tolist())):
        a, d, m = x[o:o + c].double(), dy[o:o + c].double(), w[e].double()
        check(y[o:o + c], a @ m.T, a.abs() @ m.abs().T, K, ("forward", e, c))
        check(dx[o:o + c], d @ m, d.abs() @ m.abs(), N, ("dgrad", e, c))
        check(dw[e], d.T @ a, d.abs().T @ a.abs(), max(c, 1), ("wgrad", e, c))
    return x, dy, w, count, offsets, y, dx, dw


@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 8), ([5], 64, 64), ([1, 0, 2], 128, 128), ([16, 17, 15], 72, 136), ([64, 63, 65, 0], 256, 192),
    ([127, 129, 128], 264, 320), ([300, 1, 0, 0, 31], 512, 256), ([255, 257, 256], 384, 640), ([1000], 1000, 1000),
    ([0, 0, 0], 64, 64), ([7] * 70, 96, 64), ([3, 0] * 100, 64, 40), ([33, 500, 90], 1536, 2048), ([600, 700], 24, 2048),
    ([600, 700], 2048, 24)])
def test_products_ragged(counts, N, K):
    run_all(counts, N, K)


@pytest.mark.parametrize("counts", [[40, 0, 90], [1, 1, 1], [200, 130, 64]])
def test_rows_of_no_expert_are_left_alone(counts):
    """Gaps full of NaN and infinities around every segment."""
    run_all(counts, 256, 128, gaps=5)


def test_one_token_of_many_experts():
    counts = [0] * 256
    for e in (3, 17, 64, 101, 102, 200, 254, 255):
        counts[e] = 1
    run_all(counts, 512, 768)


@pytest.mark.parametrize("counts,N,K", [([1024] * 4, 1024, 2048), ([2500, 10, 700], 1280, 768)])
def test_products_larger(counts, N, K):
    run_all(counts, N, K, seed=3)


# depths that the pairs of a cluster divide: whole and ragged stages, parts
# without a stage, odd heights, ragged ends of the summed rows, empty experts
@pytest.mark.parametrize("counts,N,K", [
    ([64], 1024, 2048), ([3], 128, 4096), ([290, 0, 291], 120, 3680), ([1], 8, 2056), ([70], 2056, 8),
    ([5003], 256, 256), ([0, 1, 2047], 64, 72), ([4096, 3], 136, 264), ([640], 40, 1160), ([33], 7168, 136),
    ([600, 601], 1032, 120), ([129, 0, 0, 1, 300], 256, 1000), ([2000], 264, 24), ([17], 520, 520), ([8191], 72, 8)])
def test_few_tiles_share_the_depth(counts, N, K):
    first = run_all(counts, N, K, seed=5)
    again = run_all(counts, N, K, seed=5)
    for x, y in zip(first[5:], again[5:]):
        assert torch.equal(x, y)
    run_all(counts, N, K, gaps=5, seed=6)


def test_segments_of_more_rows_than_there_are():
    """Overlapping segments are not allowed; here they end with an error or as written twice."""
    x, w = torch.randn(64, 2048, device="cuda").bfloat16(), torch.randn(6, 64, 2048, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    count, offsets = torch.full((6,), 64, **i32), torch.zeros(6, **i32)
    y = torch.zeros(64, 64, dtype=x.dtype, device="cuda")
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    api.moe_nvfp4_expert_linear(x, w, count, offsets, y, status[:1])
    assert api.moe_nvfp4_last_device_status(status) in (0, api.MOE_ERR_INVALID_ARG)


def test_a_neighbours_nan_stays_its_own():
    x, dy, w, count, offsets, y, dx, dw = run_all([30, 40, 50], 128, 192, poison=False)
    keep = (y.clone(), dx.clone(), dw.clone())
    x[30:70], dy[30:70] = float("nan"), float("nan")
    w[1] = float("inf")
    api.moe_nvfp4_expert_linear(x, w, count, offsets, y)
    api.moe_nvfp4_expert_linear_dgrad(dy, w, count, offsets, dx)
    api.moe_nvfp4_expert_linear_wgrad(dy, x, count, offsets, dw)
    for got, was in ((y, keep[0]), (dx, keep[1])):
        assert torch.equal(got[:30], was[:30]) and torch.equal(got[70:], was[70:])
        assert bool(torch.isnan(got[30:70].float()).all())
    assert torch.equal(dw[0], keep[2][0]) and torch.equal(dw[2], keep[2][2]) and bool(torch.isnan(dw[1].float()).all())


def test_bad_segments_count_as_empty():
    K, N, R = 64, 128, 100
    x = torch.randn(R, K, device="cuda").bfloat16()
    w = torch.randn(4, N, K, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    count, offsets = torch.tensor([10, 50, -3, 20], **i32), torch.tensor([0, 60, 10, -5], **i32)
    y = torch.full((R, N), 9.0, dtype=x.dtype, device="cuda")
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    api.moe_nvfp4_expert_linear(x, w, count, offsets, y, status[:1])
    assert bool((y[10:] == 9.0).all())
    check(y[:10], x[:10].double() @ w[0].double().T, x[:10].double().abs() @ w[0].double().abs().T, K, "kept")
    assert api.moe_nvfp4_last_device_status(status) == api.MOE_ERR_INVALID_ARG
    dw = torch.full((4, N, K), 9.0, dtype=x.dtype, device="cuda")
    api.moe_nvfp4_expert_linear_wgrad(y, x, count, offsets, dw, status[:1])
    assert not dw[1:].any()
    assert api.moe_nvfp4_last_device_status(status) == api.MOE_ERR_INVALID_ARG


def test_no_rows():
    w = torch.randn(3, 64, 32, device="cuda").bfloat16()
    count, offsets, R = segments([0, 0, 0])
    e = lambda n: torch.empty(0, n, dtype=w.dtype, device="cuda")
    api.moe_nvfp4_expert_linear(e(32), w, count, offsets, e(64))
    api.moe_nvfp4_expert_linear_dgrad(e(64), w, count, offsets, e(32))
    dw = torch.full_like(w, float("nan"))
    api.moe_nvfp4_expert_linear_wgrad(e(64), e(32), count, offsets, dw)
    assert not dw.any()


def test_gradients_against_differences():
    """L = <c, y> is linear in x and in w: the gradients' products with a
    direction equal L's differences, to the BF16 rounding of the gradients."""
    counts, N, K = [20, 0, 45, 7], 96, 64
    g = torch.Generator("cuda").manual_seed(2)
    x, c, w, count, offsets, _, dx, dw = run_all(counts, N, K, poison=False)
    def loss(x, w):
        s = 0.0
        for e, (n, o) in enumerate(zip(counts, offsets.tolist())):
            s += float(((x[o:o + n] @ w[e].T) * c[o:o + n].double()).sum())
        return s
    vx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    vw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
    x64, w64 = x.double(), w.double()
    num = (loss(x64 + vx, w64) - loss(x64 - vx, w64)) / 2
    assert abs(float((dx.double() * vx).sum()) - num) <= 2.0 ** -8 * float((dx.double() * vx).abs().sum())
    num = (loss(x64, w64 + vw) - loss(x64, w64 - vw)) / 2
    assert abs(float((dw.double() * vw).sum()) - num) <= 2.0 ** -8 * float((dw.double() * vw).abs().sum())


def test_repeatable_on_a_side_stream_and_in_a_graph():
    counts, N, K = [130, 3, 0, 290], 384, 512
    x, dy, w, count, offsets, y, dx, dw = run_all(counts, N, K, poison=False)
    keep = (y.clone(), dx.clone(), dw.clone())
    side = torch.cuda.Stream()
    def step():
        api.moe_nvfp4_expert_linear(x, w, count, offsets, y, None, side)
        api.moe_nvfp4_expert_linear_dgrad(dy, w, count, offsets, dx, None, side)
        api.moe_nvfp4_expert_linear_wgrad(dy, x, count, offsets, dw, None, side)
    torch.cuda.synchronize()
    step()
    side.synchronize()
    assert torch.equal(y, keep[0]) and torch.equal(dx, keep[1]) and torch.equal(dw, keep[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in (y, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, keep[0]) and torch.equal(dx, keep[1]) and torch.equal(dw, keep[2])


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in y, and a segment that starts beyond 2^31 elements of it."""
    R, N, K = 280000, 8192, 64
    counts = [R - 70, 70]
    count, offsets, _ = segments(counts)
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(R, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(2, N, K, generator=g, device="cuda").bfloat16()
    y = torch.empty(R, N, dtype=x.dtype, device="cuda")
    api.moe_nvfp4_expert_linear(x, w, count, offsets, y)
    for o, n, e in ((0, 64, 0), (R - 200, 130, 0), (R - 70, 70, 1)):
        a, m = x[o:o + n].double(), w[e].double()
        check(y[o:o + n], a @ m.T, a.abs() @ m.abs().T, K, o)
    dx = torch.empty_like(x)
    api.moe_nvfp4_expert_linear_dgrad(y, w, count, offsets, dx)
    o, n = R - 70, 70
    d, m = y[o:o + n].double(), w[1].double()
    check(dx[o:o + n], d @ m, d.abs() @ m.abs(), N, "dgrad")
    dw = torch.empty_like(w)
    api.moe_nvfp4_expert_linear_wgrad(y, x, count, offsets, dw)
    a = x[o:o + n].double()
    check(dw[1], d.T @ a, d.abs().T @ a.abs(), n, "wgrad")


def test_binding_refuses():
    count, offsets, R = segments([4, 4])
    x, w = torch.zeros(8, 64, device="cuda").bfloat16(), torch.zeros(2, 32, 64, device="cuda").bfloat16()
    y = torch.zeros(8, 32, device="cuda").bfloat16()
    with pytest.raises(TypeError):
        api.moe_nvfp4_expert_linear(x.float(), w, count, offsets, y)
    with pytest.raises(ValueError):
        api.moe_nvfp4_expert_linear(x[:, :32], w, count, offsets, y)
    with pytest.raises(TypeError):
        api.moe_nvfp4_expert_linear(x, w, count.long(), offsets, y)
    with pytest.raises(ValueError):
        api.moe_nvfp4_expert_linear(x, w, count[:1], offsets, y)
    with pytest.raises(api.MoEError):
        api.moe_nvfp4_expert_linear(x[:, :4].contiguous(), w[:, :, :4].contiguous(), count, offsets, y)
