"""Rates that AdamW refuses on the host, before anything is launched."""
import ctypes

import pytest

from nvfp4_mixture_experts_router_gb300 import api, build


@pytest.mark.parametrize("lr,beta1,step,ok", [(1e38, 0.9, 1, False), (1e37, 0.9, 1, False), (8e36, 0.9, 1, True), (1e30, 1 - 1e-9, 1, False),
                                              (8e37, 0.0, 1, True), (1e38, 0.0, 1, False), (8e37, 0.9, 1000, True)])
def test_rate(lr, beta1, step, ok):
    build.build()
    empty = api.moe_adamw_tensor(numel=0, param_dtype=api.MOE_DTYPE_F32, grad_dtype=api.MOE_DTYPE_F32, state_bits=32)
    rule = lambda: api.moe_adamw_rule(lr, beta1, 0.99, 1e-8, 0.0, 1.0, 1e-6, step)      # noqa: E731
    for lr_step in (None, ctypes.c_void_p(1 << 36)):        # (the host does not look at the rate of lr_step)
        want = api.MOE_OK if ok or lr_step else api.MOE_ERR_INVALID_ARG
        assert api.lib().moe_nvfp4_adamw(1, ctypes.byref(empty), rule(), None, lr_step, None) == want
