"""Experts chosen from logits, and the gradient of the logits, against plain torch
in 64 bits.  Ids are compared exactly: the choice is that of exact scores.

Bounds, with u = 2^-24.  A score e^x, x a difference of two logits: the
difference's rounding u |x|, expf 4 u, the sums and divisions after it 20 u, and
the same again for the sum that renormalizes: w is within (60 + 4 X) u of itself,
X the largest |x| among the chosen (and the sigmoid's |l|).  The softmax over all
experts takes e^x with a documented error of (3 + 1.18 |x|) 2 u; its terms
weigh |x| by p, whose mean is log E at most, and its sum has 37 additions at
most: (2 (40 + 1.2 log E) + 30 + X) u.  A gradient w (u_k - sum w u) adds the sum's
additions: 3 times that of w (|u_k| + sum w |u|), and half a unit of its type."""
import math

import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build, train

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32
SOFTMAX, SIGMOID = api.MOE_SCORE_SOFTMAX, api.MOE_SCORE_SIGMOID
MAX, TOP2 = api.MOE_GROUP_MAX, api.MOE_GROUP_TOP2
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def logit(l):
    l = l.double()
    return torch.where(l > -INF, l, -INF).clamp(max=3.4028234663852886e38)


def score(l, kind):
    if kind == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top > -INF, top, 0.0))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def chosen(logits, bias, rule, K):
    """Ids of the definition: the scores in 64 bits, stable sorts."""
    l = logit(logits)
    T, E = l.shape
    can = l > -INF
    s = score(l, rule.score)
    c = l
    if bias is not None:
        b = bias.double()
        can = can & (b > -INF)
        s = c = s + b
    c = torch.where(can, c, -INF)
    if rule.groups > 1:
        g = torch.where(can, s if rule.group_score == TOP2 else c, -INF).view(T, rule.groups, -1)
        two = g.sort(dim=2, descending=True).values
        of = two[:, :, 0]
        if rule.group_score == TOP2 and two.shape[2] > 1:
            of = of + torch.where(two[:, :, 1] > -INF, two[:, :, 1], 0.0)
        best = of.sort(dim=1, descending=True, stable=True).indices[:, :rule.topk_groups]
        keep = torch.zeros_like(of, dtype=torch.bool).scatter_(1, best, True)
        c = torch.where(keep.repeat_interleave(E // rule.groups, 1), c, -INF)
    r = c.sort(dim=1, descending=True, stable=True)
    return torch.where(r.values[:, :K] > -INF, r.indices[:, :K], -1).int()


def weights(logits, ids, rule):
    """Weights in 64 bits for given ids, and their bound's X."""
    l = logit(logits)
    at = ids.long().clamp(min=0)
    there = ids >= 0
    p = torch.where(there, l.gather(1, at), -INF)
    if rule.renormalize:
        m = p.amax(1, keepdim=True)
        m = torch.where(m > -INF, m, 0.0)
        x = p - m
        part = torch.exp(x)
        if rule.score == SIGMOID:
            part = torch.exp(p.clamp(max=0.0) - m.clamp(max=0.0)) / (1.0 + torch.exp(-p.abs()))
        w = part / part.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = score(l, rule.score).gather(1, at)
        top = l.amax(1, keepdim=True)
        x = p - torch.where(top > -INF, top, 0.0)
    X = torch.where(there, x.abs(), 0.0).amax(1, keepdim=True).clamp(max=200.0)
    return torch.where(there, w * rule.scale, 0.0), X


def units(E, X, rule):
    if rule.score == SOFTMAX and not rule.renormalize:
        return 2 * (40 + 1.2 * math.log(E)) + 30 + X
    return 60 + 4 * X


def route(logits, bias, rule, K, stream=None):
    T = logits.shape[0]
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), NAN, device="cuda")
    api.moe_nvfp4_route_topk(logits, bias, rule, ids, w, stream)
    return ids, w


def check(logits, bias, rule, K):
    ids, w = route(logits, bias, rule, K)
    want = chosen(logits, bias, rule, K)
    assert torch.equal(ids, want), f"{int((ids != want).any(1).sum())} tokens differ"
    ww, X = weights(logits, ids, rule)
    bound = units(logits.shape[1], X, rule) * U * ww.abs() + 1e-37
    err = (w.double() - ww).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    return ids, w


def normal(T, E, dt=F32, seed=0, spread=1.0):
    g = torch.Generator("cuda").manual_seed(seed * 7919 + T * 31 + E)
    return (spread * torch.randn(T, E, generator=g, device="cuda")).to(dt)


def bias_of(E, size=0.05, seed=1):
    return size * torch.randn(E, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


SHAPES = [(1, 1, 1), (3, 2, 1), (5, 7, 7), (64, 31, 5), (33, 32, 8), (200, 33, 32), (1, 256, 8), (153, 40, 3), (300, 64, 6),
          (77, 100, 9), (40, 160, 6), (1000, 256, 8), (65, 257, 4), (20, 384, 8), (19, 512, 32), (30, 513, 10), (25, 1000, 8),
          (2500, 1024, 8)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dt", [F32, BF])
def test_sizes(T, E, K, kind, biased, dt):
    for renorm in (True, False):
        rule = api.RouteRule(score=kind, renormalize=renorm, scale=1.0 if renorm else 2.5)
        check(normal(T, E, dt, spread=2.0), bias_of(E) if biased else None, rule, K)


@pytest.mark.parametrize("E,groups,top", [(256, 8, 4), (256, 8, 1), (64, 2, 1), (60, 6, 3), (60, 30, 7), (160, 8, 3), (32, 32, 9),
                                          (31, 31, 5), (1024, 32, 4), (512, 4, 2), (40, 5, 5), (96, 3, 2), (1000, 8, 4), (8, 4, 2),
                                          (1024, 2, 1)])
@pytest.mark.parametrize("group_score", [MAX, TOP2])
@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
def test_groups(E, groups, top, group_score, kind):
    K = min(8, top * (E // groups))
    rule = api.RouteRule(score=kind, groups=groups, topk_groups=top, group_score=group_score)
    for bias in (None, bias_of(E)):
        check(normal(700, E), bias, rule, K)
        check(normal(33, E, BF), bias, rule, K)


@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
def test_many_tokens(kind):
    """Enough of them that FP32 scores alone would choose otherwise somewhere."""
    rule = api.RouteRule(score=kind, groups=8, topk_groups=4, group_score=TOP2)
    check(normal(16384, 256), bias_of(256), rule, 8)
    check(normal(16384, 256), bias_of(256, 0.002), api.RouteRule(score=kind), 8)


@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("E", [8, 64, 256, 1024])
def test_near_ties(kind, E):
    """A bias that makes every expert's score the same but for the bias's own rounding."""
    base = normal(1, E, spread=1.5)
    s = score(logit(base), kind)[0]
    bias = (0.75 - s).float()
    # the same row, and rows whose logits are a unit of the last place off here and there
    g = torch.Generator("cuda").manual_seed(E)
    rows = base.repeat(50, 1)
    up = torch.rand(50, E, generator=g, device="cuda") < 0.3
    up[0] = False
    rows = torch.where(up, torch.nextafter(rows, torch.full_like(rows, INF)), rows)
    K = min(8, E // 2)
    check(rows, bias, api.RouteRule(score=kind), K)
    for gs in (MAX, TOP2):
        check(rows, bias, api.RouteRule(score=kind, groups=4, topk_groups=2, group_score=gs), min(K, E // 4))


@pytest.mark.parametrize("copies", [1, 2, 5, 40])
@pytest.mark.parametrize("K", [1, 2, 3])
def test_equal_experts_before_a_better_one(copies, K):
    """Scores that FP32 takes for equal: `copies` of one expert, which are equal exactly, and behind them one that
    is better in the thirteenth digit."""
    E = 64
    l, bias = torch.full((3, E), -50.0, device="cuda"), torch.zeros(E, device="cuda")
    for at in (3, 50):
        l[:, at:at + min(copies, E - at)], bias[at:at + min(copies, E - at)] = -30.0, 1.0
    l[:, 60], bias[60] = -28.5, 1.0
    ids, _ = check(l, bias, api.RouteRule(score=SIGMOID), K)
    assert bool((ids[:, 0] == 60).all())


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
def test_ties_go_to_the_lower_expert(kind, dt):
    E, K = 96, 6
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.25, device="cuda")):
        for rule in (api.RouteRule(score=kind), api.RouteRule(score=kind, groups=8, topk_groups=3, group_score=TOP2)):
            for v in (0.0, -3.5, 90.0):
                ids, _ = check(torch.full((5, E), v, device="cuda", dtype=dt), bias, rule, K)
                assert ids.tolist() == [list(range(K))] * 5
            check(normal(400, E, dt).round(decimals=0), bias, rule, K)
            check(torch.where(torch.arange(E, device="cuda") % 2 == 0, 0.0, -0.0).to(dt).repeat(3, 1), bias, rule, K)


@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", [F32, BF])
def test_masked_and_not_finite(kind, renorm, dt):
    E, K = 48, 5
    low = torch.finfo(dt).min
    l = normal(12, E, dt)
    l[1, :] = -INF
    l[2, 3:] = -INF
    l[3, :] = NAN
    l[4, ::2] = NAN
    l[5, 1::3] = low
    l[6, :] = low
    l[7, 7] = INF
    l[8, 7:9] = INF
    l[9, :40] = -INF
    l[10, 11] = torch.finfo(dt).max
    l[11, :47] = low
    b = bias_of(E)
    off = b.clone()
    off[5], off[6], off[9] = -INF, NAN, INF
    for bias in (None, b, off, torch.full((E,), -INF, device="cuda")):
        for groups, top, gs in ((1, 1, MAX), (8, 2, TOP2), (8, 2, MAX), (16, 3, TOP2)):
            rule = api.RouteRule(score=kind, groups=groups, topk_groups=top, group_score=gs, renormalize=renorm)
            ids, w = check(l, bias, rule, K)
            assert bool((ids[1] == -1).all()) and bool((w[1] == 0).all()) and bool((ids[3] == -1).all())
            assert bool(((w == 0) | (ids >= 0)).all())
            if renorm:
                total = w.double().sum(1)
                assert bool(((total - 1).abs()[(ids >= 0).any(1)] <= 1e-5).all())


def test_weights_do_not_underflow_together():
    l = torch.tensor([[-200.0, -201.0, -300.0, -200.5], [-1e30, -1e30, -2e30, -3e30]], device="cuda")
    ids, w = check(l, None, api.RouteRule(score=SIGMOID), 2)
    assert ids.tolist() == [[0, 3], [0, 1]] and bool(((w.sum(1) - 1).abs() < 1e-6).all())
    # far scores with a bias: equal to the last bit of 64, or told apart
    check(torch.tensor([[-90.0, -95.0, -100.0, -30.0]], device="cuda"), torch.zeros(4, device="cuda"),
          api.RouteRule(score=SIGMOID), 3)
    check(torch.tensor([[60.0, 50.0, 20.0, 16.5]], device="cuda"), torch.zeros(4, device="cuda"), api.RouteRule(score=SIGMOID), 3)


@pytest.mark.parametrize("E", [40, 64, 256])
@pytest.mark.parametrize("dt", [F32, BF])
def test_strided_rows(E, dt):
    """Columns of a wider tensor, at odd offsets, with NaN around them."""
    for wide, at in ((E + 24, 8), (E + 7, 3), (2 * E, E)):
        buf = torch.full((301, wide), NAN, dtype=dt, device="cuda")
        buf[:, at:at + E] = normal(301, E, dt)
        l = buf[:, at:at + E]
        rule = api.RouteRule(score=SIGMOID, groups=4, topk_groups=2, group_score=TOP2)
        a, wa = check(l, bias_of(E), rule, 4)
        b, wb = route(l.contiguous(), bias_of(E), rule, 4)
        assert torch.equal(a, b) and torch.equal(wa, wb)
        dw = normal(301, 4)
        keep = buf.clone()
        out = torch.full((301, E), NAN, dtype=dt, device="cuda")
        api.moe_nvfp4_route_topk_backward(l, a, dw, rule, out)
        assert torch.equal(buf.nan_to_num(7.0), keep.nan_to_num(7.0))
        api.moe_nvfp4_route_topk_backward(l, a, dw, rule, l)       # in place, the columns around untouched
        keep[:, at:at + E] = out
        assert torch.equal(buf.nan_to_num(7.0), keep.nan_to_num(7.0))


def gradient(logits, ids, dw, rule):
    """d sum(dw w) / d logits by differentiation in 64 bits, and the scale its bound goes by."""
    l = logit(logits).clamp(min=-1e30).requires_grad_(True)
    there, at = (ids >= 0) & (ids < l.shape[1]), ids.long().clamp(min=0, max=l.shape[1] - 1)
    # (renormalized, the sum over all experts drops out: left in, its rounding would be a gradient of the others)
    ls = l if rule.score == SOFTMAX and rule.renormalize else torch.log_softmax(l, 1) if rule.score == SOFTMAX else \
        torch.nn.functional.logsigmoid(l)
    p = torch.where(there, ls.gather(1, at), -1e30)
    if rule.renormalize:
        p = p - torch.logsumexp(p, 1, keepdim=True)
    w = torch.where(there, torch.exp(p) * rule.scale, 0.0)
    d, = torch.autograd.grad((w * dw.double()).sum(), l)
    uw = torch.where(there, w.detach() / rule.scale, 0.0)
    au = torch.where(there, dw.double().abs() * abs(rule.scale), 0.0)
    mean = (uw * au).sum(1, keepdim=True)
    size = torch.zeros_like(d).scatter_add_(1, at, torch.where(there, uw * (au + (mean if rule.renormalize or rule.score == SOFTMAX else 0)), 0.0))
    if rule.score == SOFTMAX and not rule.renormalize:
        size = size + score(logit(logits), SOFTMAX) * mean
    x = torch.where(there, (l.detach().gather(1, at) - l.detach().amax(1, keepdim=True)).abs(), 0.0)
    return d, size, x.amax(1, keepdim=True).clamp(max=200.0)


def check_backward(logits, ids, dw, rule):
    out = torch.full(logits.shape, NAN, dtype=logits.dtype, device="cuda")
    api.moe_nvfp4_route_topk_backward(logits, ids, dw, rule, out)
    d, size, X = gradient(logits, ids, dw, rule)
    if rule.score == SOFTMAX and not rule.renormalize:      # every expert's own |x|
        l = logit(logits)
        X = (l - l.amax(1, keepdim=True)).abs().clamp(max=200.0).nan_to_num(0.0)
        X = 3 * X
    bound = 3 * units(logits.shape[1], X, rule) * U * size + HALF[logits.dtype] * d.abs() * 1.01 + 1e-37
    err = (out.double() - d).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    return out


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", [F32, BF])
def test_backward(T, E, K, kind, renorm, dt):
    rule = api.RouteRule(score=kind, renormalize=renorm, scale=2.5)
    l = normal(T, E, dt, spread=2.0)
    ids, _ = route(l, None, rule, K)
    dw = normal(T, K, seed=3)
    a = check_backward(l, ids, dw, rule)
    assert torch.equal(a, check_backward(l, ids, dw, rule))
    if T > 2:       # some slots dropped, and a token with none
        ids[::3, 0] = -1
        ids[1] = -1
        ids[2, -1] = E
        out = check_backward(l, ids, dw, rule)
        assert not out[1].any()


@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_of_repeated_experts(kind, renorm):
    """Slots of one expert add up."""
    rule = api.RouteRule(score=kind, renormalize=renorm)
    l = normal(50, 16)
    ids = torch.randint(0, 4, (50, 6), generator=torch.Generator("cuda").manual_seed(2), device="cuda", dtype=torch.int32)
    check_backward(l, ids, normal(50, 6, seed=4), rule)


@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_with_masked_experts(kind, renorm):
    l = normal(60, 40)
    l[:, ::7] = -INF
    l[3] = -INF
    l[4, 1:] = -INF
    rule = api.RouteRule(score=kind, renormalize=renorm)
    ids, _ = route(l, None, rule, 5)
    out = check_backward(l, ids, normal(60, 5, seed=5), rule)
    assert bool((out[:, ::7] == 0).all()) and bool((out[3] == 0).all())


@pytest.mark.parametrize("kind", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_against_differences(kind, renorm):
    """Central differences of the weights in 64 bits: off by h^2 = 1e-8 and the rounding 1e-16 / h, on
    gradients of up to 1; the kernel's own error is below 1e-6 of them."""
    T, E, K, h = 6, 12, 4, 1e-4
    rule = api.RouteRule(score=kind, renormalize=renorm)
    l = normal(T, E).double()
    ids, _ = route(l.float(), None, rule, K)
    l = l.float().double()
    dw = normal(T, K, seed=6)
    out = check_backward(l.float(), ids, dw, rule)
    for e in range(E):
        step = torch.zeros(1, E, dtype=torch.float64, device="cuda")
        step[0, e] = h
        up, down = weights64(l + step, ids, rule), weights64(l - step, ids, rule)
        d = ((up - down) * dw).sum(1) / (2 * h)
        assert bool(((out[:, e] - d).abs() <= 1e-5).all())


def weights64(l, ids, rule):
    s = score(l, rule.score).gather(1, ids.long())
    return s / s.sum(1, keepdim=True) if rule.renormalize else s


def test_autograd_streams_and_graphs():
    T, E, K = 300, 64, 6
    rule = api.RouteRule(score=SIGMOID, groups=8, topk_groups=4, group_score=TOP2)
    l, bias, dw = normal(T, E), bias_of(E), normal(T, K, seed=8)
    leaf = l.clone().requires_grad_(True)
    ids, w = train.route(leaf, K, bias, rule)
    (w * dw).sum().backward()
    out = torch.empty_like(l)
    api.moe_nvfp4_route_topk_backward(l, ids, dw, rule, out)
    assert torch.equal(leaf.grad, out) and not ids.requires_grad
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ids2, w2 = torch.empty_like(ids), torch.empty(T, K, device="cuda")
    api.moe_nvfp4_route_topk(l, bias, rule, ids2, w2, side)
    side.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w.detach(), w2)
    graph = torch.cuda.CUDAGraph()
    static, o = l.clone(), torch.empty_like(l)
    with torch.cuda.graph(graph):
        api.moe_nvfp4_route_topk(static, bias, rule, ids2, w2)
        api.moe_nvfp4_route_topk_backward(static, ids2, dw, rule, o)
    for seed in (11, 12):
        static.copy_(normal(T, E, seed=seed))
        graph.replay()
        a, wa = route(static, bias, rule, K)
        assert torch.equal(ids2, a) and torch.equal(w2, wa)
        api.moe_nvfp4_route_topk_backward(static, a, dw, rule, out)
        assert torch.equal(o, out)


def test_no_tokens_and_refusals():
    rule = api.RouteRule()
    i = lambda T, K: torch.empty(T, K, dtype=torch.int32, device="cuda")      # noqa: E731
    f = lambda *s: torch.empty(*s, device="cuda")      # noqa: E731
    api.moe_nvfp4_route_topk(f(0, 8), None, rule, i(0, 2), f(0, 2))
    api.moe_nvfp4_route_topk_backward(f(0, 8), i(0, 2), f(0, 2), rule, f(0, 8))
    l = f(4, 8)
    for args in ((l.half(), None, rule, i(4, 2), f(4, 2)), (l.cpu(), None, rule, i(4, 2), f(4, 2)),
                 (l, None, rule, i(4, 2).long(), f(4, 2)), (l, f(8).bfloat16(), rule, i(4, 2), f(4, 2)),
                 (l, None, None, i(4, 2), f(4, 2)), (l, None, (0, 1), i(4, 2), f(4, 2))):
        with pytest.raises(TypeError):
            api.moe_nvfp4_route_topk(*args)
    for args in ((l.t(), None, rule, i(8, 2), f(8, 2)), (l, None, rule, i(5, 2), f(4, 2)), (l, None, rule, i(4, 2), f(4, 3)),
                 (l, f(7), rule, i(4, 2), f(4, 2)), (l[0], None, rule, i(4, 2), f(4, 2))):
        with pytest.raises(ValueError):
            api.moe_nvfp4_route_topk(*args)
    with pytest.raises(api.MoEError):
        api.moe_nvfp4_route_topk(l, None, api.RouteRule(groups=3), i(4, 2), f(4, 2))
    with pytest.raises(ValueError):
        api.moe_nvfp4_route_topk_backward(l, i(4, 2), f(4, 2), rule, f(4, 9))
    with pytest.raises(TypeError):
        api.moe_nvfp4_route_topk_backward(l, i(4, 2), f(4, 2), rule, l.bfloat16())


def test_with_the_layer_s_forward():
    """The layer on these ids and weights, against its own softmax routing: the same ids, so the same
    rows, and weights a few roundings apart (60 units of 2^-24 of them; half a unit of y's type beside)."""
    T, H, I, E, K = 64, 256, 128, 16, 4
    layer = api.MoELayer.create(T, H, I, E, K, api.MOE_W4A16)
    g = torch.Generator("cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()      # noqa: E731
    layer.prepare(r(E, 2 * I, H) * 0.05, r(E, H, I) * 0.05)
    x, l = r(T, H), normal(T, E)
    own = layer.forward(x, l)
    ids, w = route(l, None, api.RouteRule(), K)
    y = layer.forward_routed(x, ids, w)
    assert torch.equal(layer.view("topk_ids", torch.int32, T * K).view(T, K), ids)
    assert bool(((y.float() - own.float()).abs() <= 2.1 * 2.0 ** -8 * own.float().abs() + 1e-5 * own.float().abs().max()).all())


@pytest.mark.parametrize("E", [1024, 1000, 513])
@pytest.mark.parametrize("dt", [F32, BF])
def test_softmax_with_a_bias_that_nearly_ties(E, dt):
    """Flat rows, whose sums take the most roundings, and a bias that puts neighbours a few units of the scores' error
    apart, in either order."""
    g = torch.Generator("cuda").manual_seed(E)
    logits = (1e-2 * torch.randn(400, E, generator=g, device="cuda")).to(dt)
    p = torch.softmax(logits[0].double(), 0)
    units = torch.randint(-45, 46, (E,), generator=g, device="cuda").double()
    bias = (0.5 - p + units * 2.0 ** -23 / E).float()
    check(logits, bias, api.RouteRule(), 8)
    check(logits[:1].expand(300, E).contiguous(), bias, api.RouteRule(renormalize=False), 32)
