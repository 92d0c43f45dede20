"""AdamW at the ends of its documented ranges, against plain torch in 64 bits (bounds: test_adamw.py)."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build
from test_adamw import BF, F32, list_of, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


@pytest.mark.parametrize("lr", [0.0, 1e-31, 1e-3])
@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_squares_that_overflow(lr, on_device, bits):
    """A gradient of 1e20 has an infinite v: m / infinity moves nothing, whatever the rate."""
    for kind in ((F32, F32, bits, False), (BF, BF, bits, True)):
        t, = make([1000], *kind)
        t.g[300], t.g[999] = 1e20, -1e20
        at = t.w if t.w is not None else t.p
        before = at.clone()
        numbers = torch.tensor([lr, 3.0], device="cuda") if on_device else None
        api.moe_nvfp4_adamw(list_of([t]), api.AdamWRule(lr=lr, weight_decay=0.0), 3, None, numbers)
        assert torch.equal(at[[300, 999]], before[[300, 999]]) and bool(torch.isfinite(at).all())
        if lr < 1e-3:
            assert torch.equal(at, before)


TINY = 2.0 ** -126


@pytest.mark.parametrize("lr,eps", [(0.2, TINY), (0.5, TINY), (1e3, 1e-36), (1e30, 1e-8), (1e-18, 1e-8), (1e-25, 1e-8),
                                    (2e-30, 1e-8), (1e-3, 1e30), (1e-3, TINY), (1e-3, 1e-8)])
@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_rates_and_eps(lr, eps, on_device, bits):
    """From p = 0, so that every step shows: what has no gradient stays zero, the others take the formula's step, with
    eps at 2^-126 of the rate or above."""
    rule = api.AdamWRule(lr=lr, eps=eps, weight_decay=0.0)
    numbers = torch.tensor([lr, 1.0], device="cuda") if on_device else None
    if on_device:
        rule = rule._replace(lr=float(numbers[0]))
    rule = rule._replace(eps=max(eps, TINY * rule.lr / (1 - rule.beta1)))
    for kind in ((F32, F32, bits, False), (BF, BF, bits, True)):
        t, = make([3003], *kind)
        for v in (t.p, t.w, t.g[:600]) + ((t.m, t.v) if bits == 32 else (t.m.view(torch.uint8), t.v.view(torch.uint8))):
            if v is not None:
                v.zero_()
        run([t], rule, 1, None, numbers)
        at = t.w if t.w is not None else t.p
        assert not at[:600].any()
        assert bool((at[600:] != 0).sum() > 2300) and bool(torch.isfinite(at).all())


def test_rates_that_pass_the_range():
    """1e39 with beta1 = 0.9 at the first step: refused; on the device it makes NaN, never a wrong step."""
    t, = make([300], F32, F32, 32, False)
    before = t.p.clone()
    with pytest.raises(api.MoEError):
        api.moe_nvfp4_adamw(list_of([t]), api.AdamWRule(lr=1e38, eps=1e-30), 1)
    assert torch.equal(t.p, before)
    api.moe_nvfp4_adamw(list_of([t]), api.AdamWRule(eps=1e-30), 1, None, torch.tensor([1e38, 1.0], device="cuda"))
    assert bool(torch.isnan(t.p).all())
