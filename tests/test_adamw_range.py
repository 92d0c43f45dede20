"""AdamW at the ends of its documented ranges, against plain torch in 64 bits (bounds: test_adamw.py)."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build
from test_adamw import BF, F32, list_of, make

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
