"""Routes sorted by expert, dispatch, combine and their gradients, against
plain torch in 64 bits.

Bounds: orders and copies are exact.  A sum of K products in FP32, rounded
once to the output type: (K + 1) roundings of 2^-24 of the sum of the absolute
products, plus half an ulp of the result (2^-8 of it in BF16, 2^-24 in FP32).
dw sums H products: at most H + 1 roundings in any order."""
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


def i32(*shape, fill=-7):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def sort(ids, E, stream=None):
    T, K = ids.shape
    out = (i32(E), i32(E + 1), i32(T, K), i32(T * K))
    ws = torch.full((api.moe_nvfp4_sort_workspace_bytes(T, E, K),), 0xA5, dtype=torch.uint8, device="cuda")
    api.moe_nvfp4_sort_routes(E, ids, *out, ws, stream)
    return out


def sort_ref(ids, E):
    T, K = ids.shape
    flat = ids.reshape(-1).long().cpu()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    count = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)])
    used = int(offsets[E])
    row = torch.full((T * K,), -1)
    row[order[:used]] = torch.arange(used)
    route = torch.full((T * K,), -1)
    route[:used] = order[:used]
    return [v.to(torch.int32) for v in (count, offsets, row.reshape(T, K), route)]


def make_ids(T, E, K, seed, kind="random"):
    g = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    if kind == "one":
        ids.fill_(E - 1)
    elif kind == "dropped":
        ids.fill_(-1)
    elif kind == "mixed":
        bad = torch.tensor([-1, -2 ** 31, E, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        pick = torch.randint(0, 12, (T, K), generator=g, device="cuda")
        ids = torch.where(pick < 4, bad[pick.clamp(max=3)], ids)
    return ids.contiguous()


@pytest.mark.parametrize("T,E,K,kind", [
    (1, 256, 8, "random"), (1, 1, 1, "one"), (3, 5, 5, "mixed"), (33, 40, 3, "random"), (128, 8, 8, "one"),
    (1024, 64, 1, "mixed"), (1025, 64, 1, "mixed"), (511, 64, 6, "random"), (1000, 300, 32, "mixed"),
    (2049, 1024, 8, "random"), (700, 16, 4, "dropped"), (16384, 256, 8, "random"),
    (255, 9, 8, "mixed"), (257, 1024, 8, "random"), (1023, 5, 8, "mixed"), (1500, 1024, 8, "mixed"),
    (2048, 1000, 8, "one"), (40001, 1000, 7, "mixed")])
def test_sort_is_the_stable_order(T, E, K, kind):
    ids = make_ids(T, E, K, 100 + T, kind)
    for got, want in zip(sort(ids, E), sort_ref(ids, E)):
        assert torch.equal(got.cpu(), want)


def test_sort_of_no_tokens():
    ids = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    count, offsets, _, _ = sort(ids, 9)
    assert not count.any() and not offsets.any()


SHAPES = [(1, 7168, 8, 256, torch.bfloat16), (1, 1, 1, 1, torch.float32), (5, 96, 3, 8, torch.bfloat16),
          (37, 1001, 3, 40, torch.float32), (37, 1001, 5, 40, torch.bfloat16), (64, 8, 32, 64, torch.bfloat16),
          (130, 2050, 9, 12, torch.bfloat16), (257, 2048, 6, 64, torch.bfloat16), (3, 65536, 2, 4, torch.bfloat16),
          (2, 65535, 2, 4, torch.float32), (1000, 100, 8, 16, torch.float32)]


def data(T, H, K, E, dt, seed=0):
    g = torch.Generator("cuda").manual_seed(1000 + seed + T + H)
    ids = make_ids(T, E, K, seed + T, "mixed")
    count, offsets, row, route = sort(ids, E)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    return g, offsets[E:], row, route, r


def test_dispatch_all_shapes():
    for T, H, K, E, dt in SHAPES:
        g, used, row, route, r = data(T, H, K, E, dt)
        x = r(T, H)
        out = torch.full((T * K, H), float("nan"), dtype=dt, device="cuda")
        api.moe_nvfp4_dispatch(x, row, used, out)
        want = torch.where((route >= 0)[:, None], x[(route // K).clamp(min=0).long()], torch.zeros((), dtype=dt, device="cuda"))
        assert torch.equal(out, want), (T, H, K, dt)
        # without rows_used the rows that no route owns stay as they were
        out = torch.full((T * K + 3, H), 7.0, dtype=dt, device="cuda")
        api.moe_nvfp4_dispatch(x, row, None, out)
        n = int(used)
        assert torch.equal(out[:n], want[:n]) and bool((out[n:] == 7.0).all())


def reduce_ref(rows, row, w):
    """sum_k w * rows[row], and the sum of the absolute products, in 64 bits."""
    idx = row.long()
    there = idx >= 0
    v = rows.double()[idx.clamp(min=0)]
    v = torch.where(there[..., None], v * w.double()[..., None], torch.zeros((), dtype=torch.float64, device="cuda"))
    return v.sum(1), v.abs().sum(1)


def check_sum(got, want, mag, K, dt, where):
    err = (got.double() - want).abs()
    bound = HALF[dt] * want.abs() * (1 + 1e-6) + (K + 1) * U * mag + 1e-38
    assert bool((err <= bound).all()), (where, float((err / bound).max()))


def test_combine_and_dispatch_backward_all_shapes():
    for T, H, K, E, dt in SHAPES:
        g, used, row, route, r = data(T, H, K, E, dt, 7)
        o = r(T * K, H)
        o[int(used):] = float("nan")                       # rows of no route are not read
        w = torch.rand(T, K, generator=g, device="cuda")
        w = torch.where(row < 0, torch.full_like(w, float("nan")), w).contiguous()   # nor a dropped route's weight
        y = torch.full((T, H), float("nan"), dtype=dt, device="cuda")
        api.moe_nvfp4_combine(o, row, w, y)
        check_sum(y, *reduce_ref(o, row, torch.nan_to_num(w)), K, dt, ("combine", T, H, K, dt))
        api.moe_nvfp4_dispatch_backward(o, row, y.fill_(float("nan")))
        check_sum(y, *reduce_ref(o, row, torch.ones_like(w)), K, dt, ("dispatch_backward", T, H, K, dt))


def test_combine_backward_all_shapes():
    for T, H, K, E, dt in SHAPES:
        g, used, row, route, r = data(T, H, K, E, dt, 9)
        o, dy = r(T * K, H), r(T, H)
        n = int(used)
        o[n:] = float("nan")
        w = torch.rand(T, K, generator=g, device="cuda") - 0.5
        do = torch.full((T * K, H), float("nan"), dtype=dt, device="cuda")
        dw = torch.full((T, K), float("nan"), device="cuda")
        api.moe_nvfp4_combine_backward(dy, o, row, w, used, do, dw)
        rt = route[:n].long()
        want = (w.reshape(-1)[rt].double()[:, None] * dy.double()[rt // K])
        assert bool(((do[:n].double() - want).abs() <= (HALF[dt] + 2 * U) * want.abs() + 1e-38).all())
        assert not do[n:].any()
        idx = row.long()
        prod = torch.nan_to_num(o).double()[idx.clamp(min=0)] * dy.double()[:, None, :]
        prod = prod * (idx >= 0)[..., None]
        bound = (H + 1) * U * prod.abs().sum(2)
        assert bool(((dw.double() - prod.sum(2)).abs() <= bound).all()), (T, H, K, dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,pad,shift", [(256, 8, 0), (256, 3, 0), (256, 8, 1), (250, 6, 0)])
def test_strided_and_shifted_tokens(dt, H, pad, shift):
    """Token rows with a stride and a first element off the 16-byte boundary
    give the bits of contiguous ones; the gaps are left alone."""
    T, K, E = 77, 4, 9
    g, used, row, route, r = data(T, H, K, E, dt, 3)
    base = r(T * (H + pad) + shift)
    x = base[shift:].as_strided((T, H), (H + pad, 1))
    a, b = (torch.empty(T * K, H, dtype=dt, device="cuda") for _ in range(2))
    api.moe_nvfp4_dispatch(x, row, used, a)
    api.moe_nvfp4_dispatch(x.contiguous(), row, used, b)
    assert torch.equal(a, b)
    w = torch.rand(T, K, device="cuda")
    y = torch.empty(T, H, dtype=dt, device="cuda")
    api.moe_nvfp4_combine(a, row, w, y)
    hold = torch.full_like(base, 5.0)
    ys = hold[shift:].as_strided((T, H), (H + pad, 1))
    api.moe_nvfp4_combine(a, row, w, ys)
    assert torch.equal(ys, y)
    ys.fill_(5.0)
    assert bool((hold == 5.0).all())
    do1, do2, dw1, dw2 = torch.empty_like(a), torch.empty_like(a), torch.empty_like(w), torch.empty_like(w)
    api.moe_nvfp4_combine_backward(x, a, row, w, used, do1, dw1)
    api.moe_nvfp4_combine_backward(x.contiguous(), a, row, w, used, do2, dw2)
    assert torch.equal(do1, do2)
    assert torch.allclose(dw1, dw2, rtol=0, atol=2 * (H + 1) * U * H * 16)     # another order, each within its bound


def test_special_values_pass_through():
    T, H, K, E = 9, 64, 2, 4
    g, used, row, route, r = data(T, H, K, E, torch.bfloat16, 1)
    row = torch.arange(T * K, dtype=torch.int32, device="cuda").reshape(T, K).contiguous()
    x = r(T, H)
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = float("inf"), float("-inf"), float("nan"), -0.0
    out = torch.empty(T * K, H, dtype=x.dtype, device="cuda")
    api.moe_nvfp4_dispatch(x, row, None, out)
    assert torch.equal(out.view(torch.int16), x.view(torch.int16).repeat_interleave(K, 0))
    y = torch.empty_like(x)
    api.moe_nvfp4_combine(out, row, torch.full((T, K), 0.5, device="cuda"), y)
    assert torch.isinf(y[0, 0]) and torch.isinf(y[1, 1]) and torch.isnan(y[2, 2]) and torch.equal(y[4:], x[4:])


def test_gradient_against_differences():
    """L = <c, combine(dispatch(x) * s, w)> is linear in x and in w: the
    gradients' products with a direction equal L's differences."""
    T, H, K, E = 21, 48, 3, 6
    g, used, row, route, r = data(T, H, K, E, torch.float32, 5)
    x, c, w = r(T, H), r(T, H), torch.rand(T, K, generator=g, device="cuda")
    s = r(T * K, H)
    rows = torch.empty(T * K, H, device="cuda")
    def loss(x, w):
        idx = row.long()
        o = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
        n = int(used)
        o[:n] = x[route[:n].long() // K] * s.double()[:n]
        v = torch.where((idx >= 0)[..., None], o[idx.clamp(min=0)] * w[..., None], 0.0)
        return float((v.sum(1) * c.double()).sum())
    api.moe_nvfp4_dispatch(x, row, used, rows)
    o = (rows * s).contiguous()
    do, dw, dx = torch.empty_like(o), torch.empty_like(w), torch.empty_like(x)
    api.moe_nvfp4_combine_backward(c, o, row, w, used, do, dw)
    api.moe_nvfp4_dispatch_backward((do * s).contiguous(), row, dx)
    vx, vw = r(T, H).double(), r(T, K).double()
    x64, w64 = x.double(), w.double()
    num = (loss(x64 + vx, w64) - loss(x64 - vx, w64)) / 2
    assert abs(float((dx.double() * vx).sum()) - num) <= 1e-5 * float((dx.double() * vx).abs().sum())
    num = (loss(x64, w64 + vw) - loss(x64, w64 - vw)) / 2
    assert abs(float((dw.double() * vw).sum()) - num) <= 1e-5 * float((dw.double() * vw).abs().sum())


def test_side_stream_and_graph():
    T, H, K, E = 300, 512, 4, 16
    ids = make_ids(T, E, K, 1)
    x = torch.randn(T, H, device="cuda").bfloat16()
    w = torch.rand(T, K, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, y = torch.empty(T * K, H, dtype=x.dtype, device="cuda"), torch.empty_like(x)
    bufs = (i32(E), i32(E + 1), i32(T, K), i32(T * K))
    ws = torch.empty(api.moe_nvfp4_sort_workspace_bytes(T, E, K), dtype=torch.uint8, device="cuda")
    def step(stream):
        api.moe_nvfp4_sort_routes(E, ids, *bufs, ws, stream)
        api.moe_nvfp4_dispatch(x, bufs[2], bufs[1][E:], out, stream)
        api.moe_nvfp4_combine(out, bufs[2], w, y, stream)
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    y.zero_()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    ref, mag = reduce_ref(x[bufs[3].long() // K], bufs[2], w)
    check_sum(y, ref, mag, K, x.dtype, "graph")


def test_rows_of_the_allocation_free_routing():
    """row_of_route of moe_nvfp4_route_noalloc: tile-padded rows beyond T*K."""
    T, E, K, H = 50, 8, 2, 128
    logits = torch.randn(T, E, device="cuda")
    cap = api.moe_nvfp4_workspace_layout(api.shape(T, 128, 128, E, K), 0)["rows_cap"]
    out = {"topk_ids": i32(T * K), "topk_w": torch.empty(T * K, device="cuda"), "count": i32(E), "offsets": i32(E + 1),
           "padded_offsets": i32(E + 1), "row_of_route": i32(T * K), "route_of_row": i32(cap)}
    api.moe_nvfp4_route_noalloc(T, E, K, 0, logits, None, out)
    row = out["row_of_route"].reshape(T, K)
    x = torch.randn(T, H, device="cuda")
    rows = torch.full((cap, H), 3.0, device="cuda")
    api.moe_nvfp4_dispatch(x, row, out["padded_offsets"][E:], rows)
    assert int(row.max()) >= T * K
    assert torch.equal(rows[row.long()], x[:, None, :].expand(T, K, H))
    assert not rows[int(out["padded_offsets"][E]):].any()
    y = torch.empty_like(x)
    api.moe_nvfp4_combine(rows, row, out["topk_w"].reshape(T, K), y)
    check_sum(y, *reduce_ref(rows, row, out["topk_w"].reshape(T, K)), K, torch.float32, "padded")


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in the expert-ordered rows."""
    T, K, H = 330000, 1, 7168
    g = torch.Generator("cuda").manual_seed(3)
    row = torch.randperm(T, generator=g, device="cuda").to(torch.int32).reshape(T, K)
    x = torch.randn(T, 64, generator=g, device="cuda").bfloat16().repeat(1, H // 64)
    rows = torch.empty(T, H, dtype=x.dtype, device="cuda")
    api.moe_nvfp4_dispatch(x, row, None, rows)
    pick = torch.randint(0, T, (4096,), generator=g, device="cuda")
    assert torch.equal(rows[row.reshape(-1)[pick].long()], x[pick])
    y = torch.empty_like(x)
    api.moe_nvfp4_dispatch_backward(rows, row, y)
    assert torch.equal(y, x)
    w = torch.full((T, K), 2.0, device="cuda")
    dw = torch.empty_like(w)
    api.moe_nvfp4_combine_backward(x, rows, row, w, None, y, dw)
    assert torch.equal(y[row.reshape(-1)[pick].long()], x[pick] * 2)
    assert bool(((dw.reshape(-1)[pick].double() - x[pick].double().square().sum(1)).abs() <=
                 (H + 1) * U * x[pick].double().square().sum(1)).all())


def test_binding_refuses():
    ids = i32(4, 2, fill=0)
    row = i32(4, 2, fill=0)
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(TypeError):
        api.moe_nvfp4_dispatch(x.half(), row, None, torch.zeros(8, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        api.moe_nvfp4_dispatch(x, row, None, torch.zeros(8, 63, device="cuda"))
    with pytest.raises(ValueError):
        api.moe_nvfp4_dispatch(x.t(), row, None, torch.zeros(8, 4, device="cuda"))
    with pytest.raises(TypeError):
        api.moe_nvfp4_dispatch(x, row.long(), None, torch.zeros(8, 64, device="cuda"))
    with pytest.raises(api.MoEError):
        api.moe_nvfp4_dispatch(x, row[:, :1].contiguous(), None, x)
    with pytest.raises(ValueError):
        api.moe_nvfp4_sort_routes(4, ids, i32(4), i32(4), i32(4, 2), i32(8), torch.empty(256, dtype=torch.uint8, device="cuda"))
