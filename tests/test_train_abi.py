"""Training operators (moe_nvfp4_train.h), without a GPU: exported symbols,
workspace sizes, and the refusal of invalid arguments before any CUDA call."""
import ctypes
import os
import re

import pytest

from nvfp4_mixture_experts_router_gb300 import api, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_nvfp4_train.h")
BAD = api.MOE_ERR_INVALID_ARG


def P(i, off=0):
    """Distinct fake device pointers, 2^36 bytes apart (never dereferenced)."""
    return ctypes.c_void_p((i << 36) + off)


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_exports_every_declared_symbol(L):
    names = sorted(set(re.findall(r"MOE_API\s+[^;(]*?\b(moe_nvfp4_\w+)\s*\(", open(HEADER).read())))
    assert names == sorted(api.EXPORTED_TRAIN)
    for n in names:
        assert hasattr(L, n), n


def test_workspace_sizes(L):
    assert api.moe_nvfp4_sort_workspace_bytes(0, 1, 1) >= 4
    for T, E, K in [(-1, 8, 2), (1 << 23, 8, 2), (4, 0, 1), (4, 1025, 1), (4, 8, 0), (4, 8, 33), (1 << 22, 8, 32)]:
        assert api.moe_nvfp4_sort_workspace_bytes(T, E, K) == 0
    assert api.moe_nvfp4_layer_norm_workspace_bytes(0, 1) > 0
    assert api.moe_nvfp4_layer_norm_workspace_bytes(8, 0) == 0
    assert api.moe_nvfp4_layer_norm_workspace_bytes(8, 65537) == 0
    assert api.moe_nvfp4_layer_norm_workspace_bytes(-1, 8) == 0
    assert api.moe_nvfp4_grad_norm_workspace_bytes(0) > 0
    assert api.moe_nvfp4_grad_norm_workspace_bytes(-1) == 0
    assert api.moe_nvfp4_grad_norm_workspace_bytes(65537) == 0


def test_sort_refusals(L):
    f, ws = L.moe_nvfp4_sort_routes, 1 << 30
    ok = [8, 16, 2, P(1), P(2), P(3), P(4), P(5), P(6), ws, None]
    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    assert call(_0=-1) == BAD and call(_1=0) == BAD and call(_1=1025) == BAD and call(_2=33) == BAD
    for i in range(3, 9):
        assert call(**{f"_{i}": None}) == BAD
        assert call(**{f"_{i}": P(9, 2)}) == BAD
    assert call(_4=P(1)) == BAD and call(_6=P(7), _7=P(7)) == BAD     # overlaps
    assert call(_9=4) == api.MOE_ERR_WORKSPACE


def test_row_refusals(L):
    T, H, K, rows, dt = 8, 64, 2, 16, api.MOE_DTYPE_BF16
    f = L.moe_nvfp4_dispatch
    g = lambda T=T, H=H, K=K, rows=rows, dt=dt, x=P(1), xs=64, r=P(2), u=None, o=P(3): f(T, H, K, rows, dt, x, xs, r, u, o, None)
    for kw in [dict(T=-1), dict(H=0), dict(H=65537), dict(K=0), dict(K=33), dict(rows=-1), dict(rows=(1 << 27) + 1),
               dict(dt=2), dict(xs=63), dict(x=None), dict(r=None), dict(o=None), dict(x=P(1, 1)), dict(r=P(2, 2)),
               dict(u=P(4, 1)), dict(o=P(1)), dict(o=P(1, 2 * (7 * 64 + 63)))]:
        assert g(**kw) == BAD, kw
    assert g(T=0, rows=0) == api.MOE_OK          # nothing to do: no CUDA call
    c = lambda dw=P(6), do=P(5), w=P(4): L.moe_nvfp4_combine_backward(T, H, K, rows, dt, P(1), 64, P(2), P(3), w, None, do, dw, None)
    assert c(dw=None) == BAD and c(do=None) == BAD and c(w=None) == BAD and c(do=P(2)) == BAD and c(dw=P(4)) == BAD
    assert L.moe_nvfp4_combine(T, H, K, rows, dt, P(1), P(2), None, P(4), 64, None) == BAD
    assert L.moe_nvfp4_combine(T, H, K, rows, dt, P(1), P(2), P(3), P(1), 64, None) == BAD
    assert L.moe_nvfp4_combine(0, H, K, rows, dt, P(1), None, None, None, 64, None) == api.MOE_OK
    assert L.moe_nvfp4_dispatch_backward(T, H, K, rows, dt, P(1), P(2), P(3), 63, None) == BAD


def test_expert_refusals(L):
    for name in ("moe_nvfp4_expert_linear", "moe_nvfp4_expert_linear_dgrad", "moe_nvfp4_expert_linear_wgrad"):
        f = getattr(L, name)
        g = lambda rows=32, N=64, K=128, E=4, a=P(1), b=P(2), c=P(3), o=P(4), out=P(5), st=None: f(rows, N, K, E, a, b, c, o, out, st, None)
        for kw in [dict(rows=-1), dict(rows=(1 << 27) + 1), dict(N=4), dict(N=12), dict(K=7), dict(K=65544), dict(E=0),
                   dict(E=1025), dict(a=None), dict(b=None), dict(c=None), dict(o=None), dict(out=None),
                   dict(a=P(1, 8)), dict(b=P(2, 2)), dict(out=P(5, 8)), dict(c=P(3, 2)), dict(st=P(6, 1)),
                   dict(out=P(1)), dict(out=P(2)), dict(st=P(3))]:
            assert g(**kw) == BAD, (name, kw)
    assert L.moe_nvfp4_expert_linear(0, 64, 64, 2, None, P(2), P(3), P(4), None, None, None) == api.MOE_OK


def test_layer_norm_refusals(L):
    f = L.moe_nvfp4_layer_norm
    g = lambda T=4, H=64, dt=1, x=P(1), xs=64, ga=P(2), be=P(3), eps=1e-5, y=P(4), ys=64, m=P(5), r=P(6): f(T, H, dt, x, xs, ga, be, eps, y, ys, m, r, None)
    for kw in [dict(T=-1), dict(H=0), dict(H=65537), dict(dt=2), dict(xs=63), dict(ys=60), dict(x=None), dict(ga=None),
               dict(y=None), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(m=None), dict(r=None),
               dict(x=P(1, 2)), dict(ga=P(2, 2)), dict(y=P(1, 4)), dict(y=P(1), ys=65), dict(m=P(5), r=P(5)),
               dict(y=P(2))]:
        assert g(**kw) == BAD, kw
    assert g(T=0) == api.MOE_OK
    need = api.moe_nvfp4_layer_norm_workspace_bytes(4, 64)
    b = L.moe_nvfp4_layer_norm_backward
    h = lambda dy=P(1), x=P(2), ga=P(3), m=P(4), r=P(5), dx=P(6), dg=P(7), db=P(8), ws=P(9), n=need: b(4, 64, 1, dy, 64, x, 64, ga, m, r, dx, 64, dg, db, ws, n, None)
    for kw in [dict(dy=None), dict(x=None), dict(ga=None), dict(m=None), dict(r=None), dict(dx=None), dict(dg=None),
               dict(ws=None), dict(ws=P(9, 16)), dict(dx=P(1, 4)), dict(dg=P(8)), dict(dg=P(3)), dict(dx=P(9))]:
        assert h(**kw) == BAD, kw
    assert h(n=need - 1) == api.MOE_ERR_WORKSPACE


def test_grad_refusals(L):
    n = 2
    ptr = lambda *v: (ctypes.c_void_p * len(v))(*v)
    grads, out = ptr(1 << 36, 2 << 36), ptr(3 << 36, 4 << 36)
    num = lambda *v: (ctypes.c_int64 * len(v))(*v)
    dts = lambda *v: (ctypes.c_int32 * len(v))(*v)
    need = api.moe_nvfp4_grad_norm_workspace_bytes(n)
    f = L.moe_nvfp4_grad_norm
    assert f(-1, grads, num(4, 4), dts(0, 1), P(5), P(6), need, None) == BAD
    assert f(n, None, num(4, 4), dts(0, 1), P(5), P(6), need, None) == BAD
    assert f(n, grads, num(4, -4), dts(0, 1), P(5), P(6), need, None) == BAD
    assert f(n, grads, num(4, 1 << 40), dts(0, 1), P(5), P(6), need, None) == BAD
    assert f(n, grads, num(4, 4), dts(0, 2), P(5), P(6), need, None) == BAD
    assert f(n, ptr(1 << 36, (2 << 36) + 2), num(4, 4), dts(0, 1), P(5), P(6), need, None) == BAD
    assert f(n, ptr(1 << 36, None), num(4, 4), dts(0, 1), P(5), P(6), need, None) == BAD
    assert f(n, grads, num(4, 4), dts(0, 1), None, P(6), need, None) == BAD
    assert f(n, grads, num(4, 4), dts(0, 1), P(5), P(6, 64), need, None) == BAD
    assert f(n, grads, num(4, 4), dts(0, 1), P(5), P(6), need - 1, None) == api.MOE_ERR_WORKSPACE
    g = L.moe_nvfp4_grad_clip
    assert g(n, grads, None, num(4, 4), dts(0, 1), P(5), 1.0, 1e-6, None) == BAD
    assert g(n, grads, ptr(3 << 36, None), num(4, 4), dts(0, 1), P(5), 1.0, 1e-6, None) == BAD
    assert g(n, grads, out, num(4, 4), dts(0, 1), None, 1.0, 1e-6, None) == BAD
    for mx, eps in [(-1.0, 0.0), (float("nan"), 0.0), (float("inf"), 0.0), (1.0, -1.0), (1.0, float("inf"))]:
        assert g(n, grads, out, num(4, 4), dts(0, 1), P(5), mx, eps, None) == BAD
