"""Training operators without a GPU: lists of gradients on several devices and
overlaps of strided rows."""
import ctypes
import types

import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

BAD = api.MOE_ERR_INVALID_ARG


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


def test_a_list_passes_its_device_on(monkeypatch):
    """The binding compares it with the norm's (test_train_autograd.py)."""
    passed = []
    monkeypatch.setattr(api, "_native", types.SimpleNamespace(grad_norm=lambda *a: passed.append(a) or 0,
                                                              grad_clip=lambda *a: passed.append(a) or 0))
    grads = api.GradList([HereGrad("cuda:1"), HereGrad("cuda:1")])
    api.moe_nvfp4_grad_norm(grads, None, None)
    api.moe_nvfp4_grad_clip(grads, None, 1.0)
    assert [a[:2] for a in passed] == [(2, 1), (2, 1)]


def test_overlapping_strided_rows_are_refused():
    """Rows of one stride side by side in a buffer: refused where the columns
    meet, where a row reaches into the next one, and at another stride."""
    build.build()
    L = api.lib()
    at = lambda i, off=0: ctypes.c_void_p((i << 36) + off)
    f = lambda off, ys=128, H=64: L.moe_nvfp4_layer_norm(9, H, api.MOE_DTYPE_F32, at(1, 4096), 128, at(2), at(3), 1e-5,
                                                         at(1, 4096 + off), ys, None, None, None)
    for columns in (1, 63, -1, -63, 65, 127, -65, 128, -128, 256, 128 * 8 + 63):
        assert f(4 * columns) == BAD, columns
    assert f(4 * 64, ys=129) == BAD and f(4 * 64, ys=127) == BAD and f(4 * 64, ys=256) == BAD
    # statistics (one run of memory) inside the gaps of the rows
    assert L.moe_nvfp4_layer_norm(9, 64, api.MOE_DTYPE_F32, at(1), 128, at(2), at(3), 1e-5, at(4), 64, at(1, 256),
                                  at(5), None) == BAD
