"""Segments that the experts' products cannot take."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def test_more_segment_rows_than_rows_are_reported():
    """Six experts that all claim the same 64 rows: twelve tiles of 32 rows,
    where counts that add up to 64 rows give seven at most.  With the same
    weights for every expert each row has one right value."""
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(64, 2048, generator=g, device="cuda").bfloat16()
    w = torch.randn(1, 64, 2048, generator=g, device="cuda").bfloat16().repeat(6, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    count, offsets = torch.full((6,), 64, **i32), torch.zeros(6, **i32)
    y = torch.full((64, 64), float("nan"), dtype=x.dtype, device="cuda")
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    api.moe_nvfp4_expert_linear(x, w, count, offsets, y, status[:1])
    assert api.moe_nvfp4_last_device_status(status) == api.MOE_ERR_INVALID_ARG
    a, m = x.double(), w[0].double()
    want, mag = a @ m.T, a.abs() @ m.abs().T
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + (2048 + 4) * U * mag).all())


@pytest.mark.parametrize("product", ["forward", "dgrad", "wgrad"])
def test_segments_of_buffers_without_rows_are_reported(product):
    w = torch.randn(300, 16, 8, device="cuda").bfloat16()
    e = lambda n: torch.empty(0, n, dtype=w.dtype, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    count, offsets = torch.zeros(300, **i32), torch.zeros(300, **i32)
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    dw = torch.full_like(w, float("nan"))

    def call():
        if product == "forward":
            api.moe_nvfp4_expert_linear(e(8), w, count, offsets, e(16), status[:1])
        elif product == "dgrad":
            api.moe_nvfp4_expert_linear_dgrad(e(16), w, count, offsets, e(8), status[:1])
        else:
            api.moe_nvfp4_expert_linear_wgrad(e(16), e(8), count, offsets, dw, status[:1])
            assert not dw.any()
        return api.moe_nvfp4_last_device_status(status)

    assert call() == api.MOE_OK
    for entry, value in ((count, 1), (count, -1), (offsets, -4), (offsets, 5)):
        entry[299] = value
        assert call() == api.MOE_ERR_INVALID_ARG
        entry[299] = 0
    assert call() == api.MOE_OK
