"""An AdamW step against plain torch in 64 bits.

Bounds, with u = 2^-24 (FP32 arithmetic on the same inputs):
  m    6 u (b1 |m| + (1 - b1) |g|)                     (the two products, their constants, the clipping factor, the sum)
  v    10 u v                                            (as m, of terms that are not negative; g squared)
  p    the quotient m / (sqrt(v / c) + eps): 24 u of itself (sqrt and the division 2 units of the last place, the
       constants, the product) and that of m's error; then 4 u |p| and half a unit of p's type
  states of 8 bits: half a step of E4M3 (2^-4 of the value; 2^-10 of the scale at least, of a root 2^-9: none becomes
       zero), and the error above (a root: 8 u of itself)"""
import copy

import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build, train

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B = api.MOE_ADAMW_BLOCK
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


class Tensor:
    """One parameter with everything that belongs to it, and its values in 64 bits."""

    def __init__(self, n, p_dt, g_dt, bits, master, gen, shift=0, size=1e-3):
        r = lambda s=1.0: s * torch.randn(n, generator=gen, device="cuda")      # noqa: E731

        def put(v, dt):     # `shift` elements into a buffer of their own
            buf = torch.empty(n + shift, dtype=dt, device="cuda")
            buf[shift:] = v.to(dt)
            return buf[shift:]
        w = r(0.05)
        self.p, self.g = put(w, p_dt), put(r(size), g_dt)
        self.w = put(w, F32) if master else None
        m, v = r(0.3 * size), (r(size).square() * 0.1 + 0.3 * size * size)
        self.ms = self.vs = None
        if bits == 32:
            self.m, self.v = put(m, F32), put(v, F32)
        else:
            (mq, self.ms), (vq, self.vs) = quantize(m), quantize(v.sqrt())
            self.m, self.v = (put(q.view(torch.uint8), torch.uint8).view(F8) for q in (mq, vq))
        self.bits = bits

    def values(self):
        m, v = self.m.to(F32).double(), self.v.to(F32).double()
        if self.bits == 8:
            m, v = m * spread(self.ms, len(m)), (v * spread(self.vs, len(v))).square()
        return (self.w if self.w is not None else self.p).double(), self.g.double(), m, v


def spread(s, n):
    return s.double().repeat_interleave(B)[:n]


def blocks(v):
    return torch.nn.functional.pad(v, (0, -len(v) % B)).view(-1, B)


def quantize(v):
    s = blocks(v).abs().amax(1) / 448
    return (v / s.repeat_interleave(B)[:len(v)].clamp(min=1e-37)).clamp(-448, 448).to(F8), s


def list_of(tensors):
    get = lambda k: [getattr(t, k) for t in tensors]      # noqa: E731
    return api.AdamWList(get("p"), get("g"), get("m"), get("v"), get("ms"), get("vs"), get("w"))


def expect(t, rule, step, clip=1.0):
    p, g, m, v = t.values()
    g = g * clip
    m1 = rule.beta1 * m + (1 - rule.beta1) * g
    v1 = rule.beta2 * v + (1 - rule.beta2) * g * g
    dm = 6 * U * (rule.beta1 * m.abs() + (1 - rule.beta1) * g.abs()) + 1e-38
    over = (v1 / (1 - rule.beta2 ** step)).sqrt() + rule.eps
    rate = rule.lr / (1 - rule.beta1 ** step)
    move = rate * m1 / over
    p1 = p * (1 - rule.lr * rule.weight_decay) - move
    return p1, m1, v1, dm, 24 * U * move.abs() + rate * dm / over + 4 * U * p.abs()


def check(tensors, want):
    for t, (p, m, v, dm, dp) in zip(tensors, want):
        if t.w is not None:
            assert torch.equal(t.p, t.w.to(t.p.dtype))
        at, dt = (t.w, F32) if t.w is not None else (t.p, t.p.dtype)
        err, bound = (at.double() - p).abs(), dp + 1.01 * HALF[dt] * p.abs()
        assert bool((err <= bound).all()), float((err / bound).max())
        if t.bits == 32:
            assert bool(((t.m.double() - m).abs() <= dm).all())
            assert bool(((t.v.double() - v).abs() <= 10 * U * v + 1e-38).all())
            continue
        for q, s, value, off, least in ((t.m, t.ms, m, dm, 2.0 ** -10), (t.v, t.vs, v.sqrt(), 8 * U * v.sqrt(), 2.0 ** -9)):
            true = blocks(value).abs().amax(1) / 448
            slack = blocks(off).amax(1) / 448
            assert bool(((s.double() - true).abs() <= slack + 4 * U * true + 1e-45).all())
            each = spread(s, len(value))
            err = (q.to(F32).double() * each - value).abs()
            bound = torch.maximum(value.abs() * 2.0 ** -4, each * least) * 1.001 + 1.1 * off
            assert bool((err <= bound).all()), float((err / bound).max())
            if least == 2.0 ** -9:
                # (a root below 2^-63 has a square below 2^-126, which counts as zero: it was zero before its rounding)
                assert bool(((q.to(F32) > 0) | (value < 2.0 ** -63) | (each == 0)).all())


def run(tensors, rule=api.AdamWRule(), step=7, norm=None, lr_step=None, stream=None, slack=1.0):
    clip = 1.0
    if norm is not None:
        clip = min(1.0, rule.max_norm / (float(norm) + rule.clip_eps))
    want = [expect(t, rule, step, clip) for t in tensors]
    api.moe_nvfp4_adamw(list_of(tensors), rule, step, norm, lr_step, stream)
    check(tensors, want)


def make(sizes, p_dt, g_dt, bits, master, seed=0, shift=0, size=1e-3):
    gen = torch.Generator("cuda").manual_seed(seed)
    return [Tensor(n, p_dt, g_dt, bits, master, gen, shift, size) for n in sizes]


KINDS = [(F32, F32, False), (F32, BF, False), (BF, BF, False), (BF, BF, True), (BF, F32, True), (BF, F32, False)]


@pytest.mark.parametrize("p_dt,g_dt,master", KINDS)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [0, 1])
def test_sizes(p_dt, g_dt, master, bits, shift):
    sizes = [1, 2, 7, 8, 9, 255, 256, 257, 511, 2047, 2048, 2049, 8191, 8192, 8193, 20000, 100003]
    run(make(sizes, p_dt, g_dt, bits, master, shift=shift))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_of_all_kinds(bits):
    """More of them than a launch takes, empty ones between, and both kinds of states in one list."""
    ts = []
    for i, (p, g, w) in enumerate(KINDS * 3):
        ts += make([40 + i, 3000 + i, 0, 1] * 18, p, g, bits if i % 4 else 40 - bits, w, seed=i)
    assert len(ts) > 1200
    run(ts)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 384, 385])
def test_lengths_of_the_list(n):
    run(make([300 + i for i in range(n)], BF, BF, 32, True))


@pytest.mark.parametrize("rule,step", [
    (api.AdamWRule(), 1), (api.AdamWRule(lr=0.0), 1), (api.AdamWRule(0.1, 0.0, 0.0, 1e-3, 0.0), 1),
    (api.AdamWRule(1e-2, 0.95, 0.9, 1e-12, 0.5), 3), (api.AdamWRule(1e-4, 0.9, 0.9999, 1e-8, 0.1), 100000),
    (api.AdamWRule(1e-4, 0.9, 0.999, 1e-8, 0.1), 2 ** 40)])
@pytest.mark.parametrize("bits", [32, 8])
def test_numbers(rule, step, bits):
    run(make([3000], F32, F32, bits, False), rule, step)
    run(make([3000], BF, BF, bits, True), rule, step)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("norm", [0.0, 0.3, 1.0, 40.0])
def test_clipping(bits, norm):
    n = torch.tensor([norm], device="cuda")
    run(make([5000, 77], BF, BF, bits, True), api.AdamWRule(max_norm=0.5), 4, n)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite(bits):
    for bad in (NAN, float("inf")):
        t, = make([1000], F32, F32, bits, False)
        t.g[300] = bad
        keep = copy.deepcopy(t)
        api.moe_nvfp4_adamw(list_of([t]), api.AdamWRule(), 3)
        if bad != bad:
            assert bool(torch.isnan(t.p[300]))
        lo, hi = (256, 512) if bits == 8 else (300, 301)
        m = t.m.to(F32) if bits == 32 else t.m.to(F32) * spread(t.ms, 1000).float()
        assert not bool(torch.isfinite(m[lo:hi]).any())
        if bits == 8:
            assert bool(torch.isnan(m[lo:hi]).all())
        rest = torch.ones(1000, dtype=torch.bool, device="cuda")
        rest[lo:hi] = False
        assert bool(torch.isfinite(m[rest]).all()) and bool(torch.isfinite(t.p[rest]).all())
        # a norm that is NaN makes everything NaN, as clipping does; an infinite one makes the gradients zero
        t = copy.deepcopy(keep)
        t.g.zero_()
        api.moe_nvfp4_adamw(list_of([t]), api.AdamWRule(), 3, torch.full((1,), NAN, device="cuda"))
        assert bool(torch.isnan(t.p).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero_states_and_zero_gradients(bits):
    """The first step from zeros; then gradients of zero for long: states decay to zero and stay finite."""
    t, = make([5000], F32, F32, bits, False)
    for s in (t.m, t.v, t.ms, t.vs):
        if s is not None:
            s.view(torch.uint8).zero_()
    t.g[:700] = 0.0
    t.g[700:710] = 1e-25
    rule = api.AdamWRule(lr=1e-2, beta1=0.5, beta2=0.5, weight_decay=0.0)
    run([t], rule, 1)
    assert not t.m.to(F32)[:512].any() and not t.v.to(F32)[:512].any()
    t.g.zero_()
    p = t.p.clone()
    tensors = list_of([t])
    for step in range(2, 400):
        api.moe_nvfp4_adamw(tensors, rule, step)
    assert bool(torch.isfinite(t.p).all()) and bool((t.p - p).abs().max() <= 5 * rule.lr)
    if bits == 8:
        assert not t.ms.any() and not t.vs.any() and not t.m.to(F32).any() and not t.v.to(F32).any()


def test_a_root_in_8_bits_never_becomes_zero():
    """One element 2^-30 of its block's largest: its root would round to zero, and its quotient with m to lr / eps."""
    t, = make([256], F32, F32, 8, False)
    t.g.fill_(2.0 ** -30)
    t.g[0] = 1.0
    for s in (t.m, t.v, t.ms, t.vs):
        s.view(torch.uint8).zero_()
    rule = api.AdamWRule(lr=1e-3, weight_decay=0.0, eps=1e-30)
    run([t], rule, 1)
    assert int((t.v.to(F32) == 2.0 ** -9).sum()) == 255 and float(t.v.to(F32)[0]) == 448.0
    p = t.p.clone()
    run([t], rule, 2)
    assert float((t.p - p).abs().max()) <= 2e-3


@pytest.mark.parametrize("bits", [32, 8])
def test_outside_stays(bits):
    """Tensors inside larger buffers: what lies around them is left as it was."""
    gen = torch.Generator("cuda").manual_seed(4)
    for n in (100, 1000, 8200):
        t = Tensor(n, BF, BF, bits, True, gen)
        new = {}
        for k in ("p", "w", "m", "v", "ms", "vs"):
            v = getattr(t, k)
            if v is None:
                continue
            raw = v.view(torch.uint8)
            buf = torch.full((len(raw) + 128,), 0x5A, dtype=torch.uint8, device="cuda")
            buf[64:-64] = raw
            new[k] = buf
            setattr(t, k, buf[64:-64].view(v.dtype))
        run([t])
        for k, buf in new.items():
            assert bool((buf[:64] == 0x5A).all()) and bool((buf[-64:] == 0x5A).all()), k


def test_repeatable_on_side_streams():
    a, b = (make([30000, 5, 700], BF, BF, 8, True, seed=3) for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    api.moe_nvfp4_adamw(list_of(a), api.AdamWRule(), 5)
    api.moe_nvfp4_adamw(list_of(b), api.AdamWRule(), 5, None, None, side)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        for k in ("p", "w", "m", "v", "ms", "vs"):
            assert torch.equal(getattr(x, k).view(torch.uint8), getattr(y, k).view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_numbers_on_the_device(bits):
    """lr and t from the device, replayed from a graph: the corrections are FP32 then, each within 8 u."""
    rule = api.AdamWRule(lr=5.0, beta2=0.99)
    ts = make([3000, 40], BF, BF, bits, True)
    lr_step = torch.tensor([1e-3, 3.0], device="cuda")
    tensors = list_of(ts)
    api.moe_nvfp4_adamw(api.AdamWList([], [], [], []), rule, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_nvfp4_adamw(tensors, rule, 0, None, lr_step)
    for lr, step in ((1e-3, 3), (2e-4, 17), (2e-4, 5000)):
        lr_step.copy_(torch.tensor([lr, float(step)]))
        r = rule._replace(lr=float(lr_step[0]))
        want = [expect(t, r, step) for t in ts]
        graph.replay()
        check(ts, want)


def test_more_than_2_31_elements():
    n = 2 ** 31 + 4099
    p = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[:3], g[-5:], g[2 ** 31 - 1:2 ** 31 + 1] = 1.0, -1.0, 1.0
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // B), device="cuda") for _ in range(2))
    api.moe_nvfp4_adamw(api.AdamWList([p], [g], [m], [v], [ms], [vs]), api.AdamWRule(lr=0.25, weight_decay=0.0), 1)
    assert int((p != 0).sum()) == 10 and bool((p[:3] == -0.25).all()) and bool((p[-5:] == 0.25).all())
    assert bool((p[2 ** 31 - 1:2 ** 31 + 1] == -0.25).all()) and int((m.view(torch.uint8) != 0).sum()) == 10


# ---- train.AdamW ----------------------------------------------------------------------------

def model(seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda dt, *s: torch.nn.Parameter(torch.randn(*s, generator=g, device="cuda").to(dt))      # noqa: E731
    return [r(BF, 40, 300), r(F32, 17), r(BF, 5), r(F32, 64, 64), r(BF, 33, 7)]


def give_grads(params, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    for i, p in enumerate(params):
        p.grad = None if i == 4 or (i == 2 and seed in (0, 1, 5)) else \
            torch.randn(p.shape, generator=g, device="cuda").to(p.dtype)      # (one never, one now and then)
    if seed % 2:
        params[0].grad = torch.randn(300, 40, generator=g, device="cuda").to(BF).t()      # another order of strides


def test_optimizer_follows_torch():
    """Twelve steps beside torch's AdamW on FP32 copies with the same (clipped) gradients: a step's error is that of
    the bounds above, 40 u of an update of lr and 8 u of p, and they add up over the steps."""
    params = model()
    twin = [torch.nn.Parameter(p.detach().double()) for p in params]
    opt = train.AdamW(params, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1)
    ref = torch.optim.AdamW(twin, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, foreach=False)
    for step in range(12):
        opt.zero_grad()
        give_grads(params, step)
        norm = train.grad_norm(params)
        total = torch.cat([p.grad.double().reshape(-1) for p in params if p.grad is not None]).norm()
        assert abs(float(norm) - float(total)) <= 1e-5 * float(total)
        clip = min(1.0, 10.0 / (float(norm) + 1e-6))
        for p, t in zip(params, twin):
            t.grad = None if p.grad is None else p.grad.double() * clip
        opt.step(norm=norm, max_norm=10.0)
        ref.step()
    last = model()[4]
    assert torch.equal(params[4], last)
    for p, t, s in zip(params, twin, opt.state):
        at = s["master"].view(p.shape).double() if "master" in s else p.detach().double()
        assert bool(((at - t).abs() <= 12 * (60 * U * 1e-2 + 8 * U * t.abs())).all()), float((at - t).abs().max())


def test_optimizer_saves_and_loads():
    for bits in (32, 8):
        a, b = model(), model()
        x, y = train.AdamW(a, state_bits=bits, min_8bit=1000), train.AdamW(b, state_bits=bits, min_8bit=1000)
        kinds = [s["exp_avg"].dtype for s in x.state]
        assert kinds == [F8 if bits == 8 and p.numel() >= 1000 else F32 for p in a]
        for step in range(3):
            give_grads(a, step)
            x.step()
        saved = copy.deepcopy(x.state_dict())
        with torch.no_grad():
            for p, q in zip(a, b):
                q.copy_(p)
        y.load_state_dict(saved)
        for o, ps in ((x, a), (y, b)):
            give_grads(ps, 9)
            o.step()
        assert all(torch.equal(p, q) for p, q in zip(a, b)) and x.steps == y.steps == [4, 4, 2, 4, 0]
        with pytest.raises(ValueError):
            train.AdamW(model()[:2]).load_state_dict(saved)


def test_capturable_parameters_count_together():
    params = model()
    opt = train.AdamW(params, capturable=True)
    give_grads(params, 0)
    opt.step()
    give_grads(params, 2)       # one more has a gradient now
    with pytest.raises(ValueError):
        opt.step()


@pytest.mark.parametrize("lr", [1e-39, 1e-31, 1e-25])
def test_tiny_rates(lr):
    """A rate below 1e-30 counts as zero; above it the step is what it is."""
    t, = make([600], F32, F32, 32, False)
    t.v[:100] = 0.0
    t.g[:100] = 0.0
    p = t.p.clone()
    api.moe_nvfp4_adamw(list_of([t]), api.AdamWRule(lr=lr, weight_decay=0.0), 3)
    assert torch.equal(t.p, p) and bool(torch.isfinite(t.p).all())


def test_optimizer_in_a_graph():
    """A captured step, replayed, beside the same steps one by one with the numbers on the device."""
    a, b = model(), model()
    x, y = (train.AdamW(p, lr=1e-2, state_bits=8, min_8bit=1000, capturable=True) for p in (a, b))
    for p in a + b:
        p.grad = torch.zeros_like(p)
    for o in (x, y):
        o.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.step()
    for step in range(4):
        for ps in (a, b):
            g = torch.Generator("cuda").manual_seed(step)
            for p in ps:
                p.grad.copy_(torch.randn(p.shape, generator=g, device="cuda"))
        graph.replay()
        y.step()
    assert set(x.state_dict()["steps"]) == {5} and all(torch.equal(p, q) for p, q in zip(a, b))


def test_optimizer_without_gradients_and_wrong_arguments():
    params = model()
    opt = train.AdamW(params)
    opt.step()
    assert all(torch.equal(p, q) for p, q in zip(params, model()))
    with pytest.raises(ValueError):
        train.AdamW(params, state_bits=16)
    with pytest.raises(ValueError):
        t, = make([10], F32, F32, 32, False)
        tensors = list_of([t])
        tensors.index = 1
        api.moe_nvfp4_adamw(tensors, api.AdamWRule(), 1)
    with pytest.raises(TypeError):
        api.moe_nvfp4_adamw(list_of([t]), (1.0, 2.0), 1)
    with pytest.raises(api.MoEError):
        api.moe_nvfp4_adamw(list_of([t]), api.AdamWRule(), 0)
    twice = torch.nn.Parameter(torch.zeros(8, device="cuda"))
    twice.grad = torch.zeros_like(twice)
    with pytest.raises(ValueError):
        train.AdamW([twice, twice]).step()
