"""Routing, RMS norm and AdamW (moe_nvfp4_train.h) without a GPU: the refusal of
invalid arguments before any CUDA call, and lists that cannot be built."""
import ctypes

import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

BAD, OK = api.MOE_ERR_INVALID_ARG, api.MOE_OK
BF, F32 = api.MOE_DTYPE_BF16, api.MOE_DTYPE_F32
INF, NAN = float("inf"), float("nan")


def P(i, off=0):
    """Distinct fake device pointers, 2^36 bytes apart (never dereferenced)."""
    return ctypes.c_void_p((i << 36) + off)


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def rule(score=0, groups=1, topk_groups=1, group_score=0, renormalize=1, scale=1.0):
    return api.moe_route_rule(score, groups, topk_groups, group_score, renormalize, scale)


BAD_ROUTES = [dict(T=-1), dict(T=(1 << 22) + 1), dict(E=0), dict(E=1025), dict(K=0), dict(K=33, E=64), dict(K=17),
              dict(dt=2), dict(stride=15), dict(stride=1 << 41), dict(r=rule(score=2)), dict(r=rule(score=-1)),
              dict(r=rule(group_score=2)), dict(r=rule(groups=0)), dict(r=rule(groups=3)), dict(r=rule(groups=33), E=33),
              dict(r=rule(groups=4, topk_groups=0)), dict(r=rule(groups=4, topk_groups=5)),
              dict(r=rule(groups=8, topk_groups=1), K=3), dict(r=rule(renormalize=2)), dict(r=rule(scale=INF)),
              dict(r=rule(scale=NAN)), dict(l=None), dict(l=P(1, 2)), dict(ids=None), dict(ids=P(2, 1)),
              dict(w=None), dict(w=P(3, 2))]


@pytest.mark.parametrize("kw", BAD_ROUTES + [dict(bias=P(4, 2)), dict(ids=P(1)), dict(w=P(2)), dict(w=P(4), bias=P(4))])
def test_route_refusals(L, kw):
    a = dict(T=8, E=16, K=4, dt=F32, l=P(1), stride=None, bias=None, r=rule(), ids=P(2), w=P(3))
    a.update(kw)
    assert L.moe_nvfp4_route_topk(a["T"], a["E"], a["K"], a["dt"], a["l"], a["stride"] or max(a["E"], 1), a["bias"], a["r"],
                                  a["ids"], a["w"], None) == BAD


@pytest.mark.parametrize("kw", BAD_ROUTES + [dict(ds=15), dict(d=None), dict(d=P(4, 2)), dict(d=P(2)), dict(d=P(3)),
                                             dict(d=P(1, 4)), dict(d=P(1), ds=17)])
def test_route_backward_refusals(L, kw):
    a = dict(T=8, E=16, K=4, dt=F32, l=P(1), stride=None, r=rule(), ids=P(2), w=P(3), d=P(4), ds=None)
    a.update(kw)
    assert L.moe_nvfp4_route_topk_backward(a["T"], a["E"], a["K"], a["dt"], a["l"], a["stride"] or max(a["E"], 1), a["ids"],
                                           a["w"], a["r"], a["d"], a["ds"] or max(a["E"], 1), None) == BAD


def test_no_tokens_is_no_cuda_call(L):
    assert L.moe_nvfp4_route_topk(0, 16, 4, F32, None, 16, None, rule(), None, None, None) == OK
    assert L.moe_nvfp4_route_topk_backward(0, 16, 4, F32, None, 16, None, None, rule(), None, 16, None) == OK
    assert L.moe_nvfp4_rms_norm(0, 64, BF, None, 64, None, 0, P(3), 1e-6, None, 0, None, 0, None, None, 0, None, None) == OK
    r = api.moe_adamw_rule(1e-3, 0.9, 0.99, 1e-8, 0.0, 1.0, 1e-6, 1)
    assert L.moe_nvfp4_adamw(0, None, r, None, None, None) == OK
    empty = api.moe_adamw_tensor(numel=0, param_dtype=BF, grad_dtype=BF, state_bits=8)
    assert L.moe_nvfp4_adamw(1, ctypes.byref(empty), r, None, None, None) == OK


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(H=65537), dict(dt=2), dict(xs=63), dict(x=None), dict(x=P(1, 1)), dict(g=None),
    dict(g=P(3, 2)), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(y=None), dict(ys=63), dict(y=P(5, 1)),
    dict(res=None), dict(rs=63), dict(res=P(2, 1)), dict(hs=63), dict(h=P(4, 1)),
    dict(q=P(6)), dict(s=P(7)), dict(q=P(6), s=P(7), mode=3), dict(q=P(6), s=P(7), mode=-1), dict(q=P(6), s=P(7, 2)),
    dict(q=P(6), s=P(7, 2), mode=1), dict(rstd=P(8, 2)),
    # overlaps: h or y beside their input's start or at another stride, over one another, over the parameters
    dict(h=P(1, 64)), dict(h=P(1), hs=65), dict(y=P(2, 64)), dict(y=P(4)), dict(h=P(1), y=P(1)), dict(y=P(3)),
    dict(q=P(4), s=P(7)), dict(q=P(1), s=P(7)), dict(q=P(6), s=P(6)), dict(rstd=P(5)), dict(q=P(6), s=P(7), rstd=P(7))])
def test_rms_refusals(L, kw):
    a = dict(T=8, H=64, dt=BF, x=P(1), xs=64, res=P(2), rs=64, g=P(3), eps=1e-6, h=P(4), hs=64, y=P(5), ys=64, q=None,
             s=None, mode=0, rstd=None)
    a.update(kw)
    assert L.moe_nvfp4_rms_norm(*a.values(), None) == BAD


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(dt=2), dict(dys=63), dict(dhs=63), dict(hs=63), dict(dxs=63), dict(dy=None), dict(h=None),
    dict(g=None), dict(rstd=None), dict(dx=None), dict(dg=None), dict(ws=None), dict(ws=P(8, 16)), dict(dy=P(1, 1)),
    dict(dh=P(2, 1)), dict(dx=P(1, 64)), dict(dx=P(3), dxs=65), dict(dg=P(1)), dict(dg=P(6)), dict(dx=P(4)), dict(ws=P(7))])
def test_rms_backward_refusals(L, kw):
    a = dict(T=8, H=64, dt=BF, dy=P(1), dys=64, dh=P(2), dhs=64, h=P(3), hs=64, g=P(4), rstd=P(5), dx=P(6), dxs=64, dg=P(7),
             ws=P(8), n=1 << 30)
    a.update(kw)
    assert L.moe_nvfp4_rms_norm_backward(*a.values(), None) == BAD


def test_rms_workspace(L):
    assert api.moe_nvfp4_rms_norm_workspace_bytes(0, 1) > 0
    for T, H in ((-1, 8), (8, 0), (8, 65537), ((1 << 22) + 1, 8)):
        assert api.moe_nvfp4_rms_norm_workspace_bytes(T, H) == 0
    need = api.moe_nvfp4_rms_norm_workspace_bytes(8, 64)
    assert L.moe_nvfp4_rms_norm_backward(8, 64, BF, P(1), 64, None, 0, P(3), 64, P(4), P(5), P(6), 64, P(7), P(8), need - 1,
                                         None) == api.MOE_ERR_WORKSPACE


def test_adamw_refusals(L):
    def tensor(**kw):
        t = dict(param=1 << 36, grad=2 << 36, exp_avg=3 << 36, exp_avg_sq=4 << 36, exp_avg_scale=None,
                 exp_avg_sq_scale=None, master=None, numel=100, param_dtype=F32, grad_dtype=F32, state_bits=32, reserved=0)
        t.update(kw)
        return api.moe_adamw_tensor(**t)

    def call(t=None, n=1, norm=None, lr_step=None, **kw):
        r = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, max_norm=1.0, clip_eps=1e-6, step=1)
        r.update(kw)
        return L.moe_nvfp4_adamw(n, ctypes.byref(t) if t is not None else None, api.moe_adamw_rule(**r), norm, lr_step, None)

    e = 1 << 36
    for kw in (dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param=e + 2),
               dict(grad=e + 1), dict(exp_avg=e + 2), dict(exp_avg_sq=e + 2), dict(numel=-1), dict(numel=1 << 40),
               dict(param_dtype=2), dict(grad_dtype=-1), dict(state_bits=16), dict(state_bits=0), dict(reserved=1),
               dict(exp_avg_scale=5 << 36), dict(exp_avg_sq_scale=5 << 36), dict(master=5 << 36),
               dict(param_dtype=BF, master=e + 2), dict(state_bits=8), dict(state_bits=8, exp_avg_scale=5 << 36),
               dict(state_bits=8, exp_avg_scale=5 << 36, exp_avg_sq_scale=e + 2)):
        assert call(tensor(**kw)) == BAD, kw
    assert call(None) == BAD and call(tensor(), n=-1) == BAD and call(tensor(), n=65537) == BAD
    for kw in (dict(lr=-1.0), dict(lr=NAN), dict(lr=INF), dict(lr=1e39), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=NAN),
               dict(beta2=1.0), dict(beta2=NAN), dict(eps=0.0), dict(eps=1e-60), dict(eps=INF), dict(eps=NAN),
               dict(weight_decay=-0.1), dict(weight_decay=NAN), dict(step=0), dict(step=-1),
               dict(norm=P(9), max_norm=-1.0), dict(norm=P(9), max_norm=NAN), dict(norm=P(9), clip_eps=INF),
               dict(norm=P(9, 2)), dict(lr_step=P(9, 2))):
        assert call(tensor(), **kw) == BAD, kw


class Fake:
    """What a list reads of a CUDA tensor, on a device that need not exist."""
    is_cuda = True

    def __init__(self, numel=300, dtype=torch.float32, device="cuda:0", at=0, contiguous=True):
        self.dtype, self.device, self._n, self._at, self._c = dtype, torch.device(device), numel, at, contiguous

    def numel(self):
        return self._n

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return self._at


def test_lists_that_cannot_be_built():
    f8, bf, F = torch.float8_e4m3fn, torch.bfloat16, Fake
    ok = lambda **k: api.AdamWList(**{**dict(params=[F()], grads=[F()], exp_avg=[F()], exp_avg_sq=[F()]), **k})   # noqa: E731
    assert ok().n == 1
    assert ok(exp_avg=[F(dtype=f8)], exp_avg_sq=[F(dtype=f8)], exp_avg_scale=[F(2)], exp_avg_sq_scale=[F(2)]).n == 1
    for kw in (dict(grads=[F(dtype=torch.float16)]), dict(params=[F(dtype=torch.float16)]), dict(exp_avg=[F(dtype=bf)]),
               dict(exp_avg=[F(dtype=f8)]), dict(master=[F()]), dict(params=[F(dtype=bf)], master=[F(dtype=bf)])):
        with pytest.raises(TypeError):
            ok(**kw)
    for kw in (dict(grads=[]), dict(exp_avg=[]), dict(master=[]), dict(grads=[F(299)]), dict(exp_avg=[F(301)]),
               dict(grads=[F(contiguous=False)]), dict(params=[F(contiguous=False)]), dict(exp_avg_sq=[F(contiguous=False)]),
               dict(grads=[F(device="cuda:1")]), dict(exp_avg=[F(device="cuda:1")]), dict(exp_avg_scale=[F(2)]),
               dict(exp_avg=[F(dtype=f8)], exp_avg_sq=[F(dtype=f8)]),
               dict(exp_avg=[F(dtype=f8)], exp_avg_sq=[F(dtype=f8)], exp_avg_scale=[F(1)], exp_avg_sq_scale=[F(2)]),
               dict(params=[F(at=64), F(at=64)], grads=[F(), F()], exp_avg=[F(), F()], exp_avg_sq=[F(), F()])):
        with pytest.raises(ValueError):
            ok(**kw)


def test_structures_have_the_header_s_size():
    assert ctypes.sizeof(api.moe_route_rule) == 24
    assert ctypes.sizeof(api.moe_adamw_tensor) == 80
    assert ctypes.sizeof(api.moe_adamw_rule) == 64
