"""Training operators without a GPU: lists of gradients on several devices."""
import types

import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api


class FakeGrad:
    """What a list reads of a CUDA tensor, on a device that need not exist."""
    dtype, is_cuda = torch.float32, True

    def __init__(self, device, numel=8):
        self.device, self._numel = torch.device(device), numel

    def numel(self):
        return self._numel

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("the address of a tensor on another device was read")


class HereGrad(FakeGrad):
    def data_ptr(self):
        return 1 << 36


def test_gradients_on_two_devices_are_refused():
    with pytest.raises(ValueError, match="device"):
        api.GradList([HereGrad("cuda:0"), FakeGrad("cuda:1")])
    with pytest.raises(ValueError, match="device"):
        api.GradList([HereGrad("cuda:0")], [FakeGrad("cuda:1")])
    with pytest.raises(ValueError, match="device"):
        api.GradList([HereGrad("cuda:0"), FakeGrad("cuda:1", numel=0)])


def test_a_list_of_another_device_than_the_norm_is_refused(monkeypatch):
    launched = []
    monkeypatch.setattr(api, "_native", types.SimpleNamespace(grad_norm=lambda *a: launched.append(a) or 0,
                                                              grad_clip=lambda *a: launched.append(a) or 0))
    grads = api.GradList([HereGrad("cuda:1"), HereGrad("cuda:1")])
    here, there = FakeGrad("cuda:0"), FakeGrad("cuda:1")
    with pytest.raises(ValueError, match="device"):
        api.moe_nvfp4_grad_norm(grads, here, None)
    with pytest.raises(ValueError, match="device"):
        api.moe_nvfp4_grad_clip(grads, here, 1.0)
    assert not launched
    api.moe_nvfp4_grad_norm(grads, there, None)
    api.moe_nvfp4_grad_clip(grads, there, 1.0)
    api.moe_nvfp4_grad_norm(api.GradList([]), here, None)      # an empty list is on no device
    assert len(launched) == 3
