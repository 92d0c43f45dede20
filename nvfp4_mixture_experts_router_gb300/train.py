"""The training operators as differentiable torch functions.

Each function allocates its outputs and workspaces with torch, runs on the
current stream, and has its gradient from the same library (api.py has the
calls themselves, on the caller's buffers).  A pre-norm Mixture-of-Experts
block, with the router and the activation in torch:

    h = train.layer_norm(x, gamma, beta)
    ids, w = top-K of the router's logits of h          # [T, K]
    routes = train.sort_routes(ids, E)
    z = train.expert_linear(train.dispatch(h, routes), w1, routes)
    o = train.expert_linear(activation(z), w2, routes)
    y = x + train.combine(o, routes, w)

examples/moe_block.py trains one.
"""
from __future__ import annotations

from dataclasses import dataclass
from functools import cached_property
from typing import Iterable, Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import api


@dataclass
class Routes:
    """The routes of T tokens sorted by expert (moe_nvfp4_sort_routes)."""
    E: int
    count: torch.Tensor         # int32 [E]
    offsets: torch.Tensor       # int32 [E + 1]
    row_of_route: torch.Tensor  # int32 [T, K], -1: dropped
    route_of_row: torch.Tensor  # int32 [T * K], -1: no route
    status: Optional[torch.Tensor] = None   # int32 [1]: errors that the device's products found

    @property
    def rows(self) -> int:
        return self.route_of_row.shape[0]

    @cached_property
    def used(self) -> torch.Tensor:
        """The number of kept routes, one device int32."""
        return self.offsets[self.E:]

    def check(self) -> None:
        """Waits for the current stream and raises MoEError if an experts' product
        or a gradient of one, on these or other routes of the device, has found a
        segment outside its rows (MOE_ERR_INVALID_ARG) or given up a wait
        (MOE_ERR_TIMEOUT: its output is undefined) since the last error was raised."""
        if self.status is not None and int(self.status) != 0:
            raise api.MoEError("an experts' product", api.moe_nvfp4_last_device_status(self.status))


_status_words = {}


def _status_word(device: torch.device) -> torch.Tensor:
    """The device's status word for the products of this module.  One for all
    routes: a word each cost the sort a launch to clear it (16 -> 32 us of host
    time)."""
    word = _status_words.get(device)
    if word is None:
        word = torch.zeros(1, dtype=torch.int32, device=device)
        if not torch.cuda.is_current_stream_capturing():    # else it is the graph's, cleared by its replays
            torch.cuda.current_stream(device).synchronize() # other streams use it too
            word = _status_words.setdefault(device, word)
    return word


def sort_routes(topk_ids: torch.Tensor, E: int) -> Routes:
    """Routes of topk_ids [T, K] (int32; ids outside [0, E) are dropped).  Errors
    that the experts' products find on the device are read with Routes.check."""
    T, K = topk_ids.shape
    i32 = dict(dtype=torch.int32, device=topk_ids.device)
    r = Routes(E, torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T, K, **i32),
               torch.empty(T * K, **i32))
    nbytes = api.moe_nvfp4_sort_workspace_bytes(T, E, K)
    if nbytes == 0:
        raise api.MoEError("moe_nvfp4_sort_workspace_bytes", api.MOE_ERR_INVALID_ARG)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=topk_ids.device)
    api.moe_nvfp4_sort_routes(E, topk_ids, r.count, r.offsets, r.row_of_route, r.route_of_row, ws)
    r.status = _status_word(topk_ids.device)
    return r


def _check_rows(rows: torch.Tensor, routes: Routes, name: str) -> None:
    """The library takes a route outside its buffer for a dropped one, and a
    segment outside it for an empty one."""
    if rows.shape[0] < routes.rows:
        raise ValueError(f"{name} has {rows.shape[0]} rows for {routes.rows} routes")


def _clear_tail(rows: torch.Tensor, routes: Routes) -> torch.Tensor:
    """Zeros in the rows past the kept routes (a dispatch of no tokens)."""
    api.moe_nvfp4_dispatch(None, None, routes.used, rows)
    return rows


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps):
        T = x.shape[0]
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        mean, rstd = (torch.empty(T, dtype=torch.float32, device=x.device) for _ in range(2))
        api.moe_nvfp4_layer_norm(x, gamma, beta, eps, y, mean, rstd)
        ctx.save_for_backward(x, gamma, mean, rstd)
        ctx.with_beta = beta is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, gamma, mean, rstd = ctx.saved_tensors
        dy = dy.contiguous()
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dgamma = torch.empty_like(gamma)
        dbeta = torch.empty_like(gamma) if ctx.with_beta else None
        ws = torch.empty(api.moe_nvfp4_layer_norm_workspace_bytes(*x.shape), dtype=torch.uint8, device=x.device)
        api.moe_nvfp4_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws)
        return dx, dgamma, dbeta, None


def layer_norm(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of x [T, H] (BF16 or FP32); gamma and beta [H] FP32."""
    return _LayerNorm.apply(x, gamma, beta, eps)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, routes):
        ctx.routes, ctx.shape = routes, x.shape
        rows = torch.empty(routes.rows, x.shape[1], dtype=x.dtype, device=x.device)
        api.moe_nvfp4_dispatch(x, routes.row_of_route, routes.used, rows)
        return rows

    @staticmethod
    @once_differentiable
    def backward(ctx, drows):
        dx = torch.empty(ctx.shape, dtype=drows.dtype, device=drows.device)
        api.moe_nvfp4_dispatch_backward(drows.contiguous(), ctx.routes.row_of_route, dx)
        return dx, None


def dispatch(x: torch.Tensor, routes: Routes) -> torch.Tensor:
    """The tokens' rows in the order of the experts, [T * K, H]; zeros past the kept routes."""
    return _Dispatch.apply(x, routes)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o_rows, routes, topk_w):
        ctx.routes = routes
        ctx.save_for_backward(o_rows, topk_w)
        y = torch.empty(topk_w.shape[0], o_rows.shape[1], dtype=o_rows.dtype, device=o_rows.device)
        api.moe_nvfp4_combine(o_rows, routes.row_of_route, topk_w, y)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        o_rows, topk_w = ctx.saved_tensors
        do, dw = torch.empty_like(o_rows), torch.empty_like(topk_w)
        api.moe_nvfp4_combine_backward(dy.contiguous(), o_rows, ctx.routes.row_of_route, topk_w, ctx.routes.used, do,
                                       dw)
        return do, None, dw


def combine(o_rows: torch.Tensor, routes: Routes, topk_w: torch.Tensor) -> torch.Tensor:
    """The tokens' sums of their routes' rows times topk_w [T, K] FP32."""
    _check_rows(o_rows, routes, "o_rows")
    return _Combine.apply(o_rows.contiguous(), routes, topk_w.contiguous())


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x_rows, w, routes):
        ctx.routes = routes
        ctx.save_for_backward(x_rows, w)
        y = torch.empty(x_rows.shape[0], w.shape[1], dtype=w.dtype, device=w.device)
        api.moe_nvfp4_expert_linear(x_rows, w, routes.count, routes.offsets, y, routes.status)
        return _clear_tail(y, routes)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x_rows, w = ctx.saved_tensors
        r, dy = ctx.routes, dy.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = torch.empty_like(x_rows)
            api.moe_nvfp4_expert_linear_dgrad(dy, w, r.count, r.offsets, dx, r.status)
            _clear_tail(dx, r)
        if ctx.needs_input_grad[1]:
            dw = torch.empty_like(w)
            api.moe_nvfp4_expert_linear_wgrad(dy, x_rows, r.count, r.offsets, dw, r.status)
        return dx, dw, None


def expert_linear(x_rows: torch.Tensor, w: torch.Tensor, routes: Routes) -> torch.Tensor:
    """Every expert's rows times its matrix: x_rows [rows, K], w [E, N, K], BF16;
    zeros past the kept routes, in the gradient of x_rows too, so that sums over
    all rows (of a bias after it, say) count the routes alone."""
    _check_rows(x_rows, routes, "x_rows")
    return _ExpertLinear.apply(x_rows.contiguous(), w, routes)


def clip_grad_norm_(parameters: Union[torch.Tensor, Iterable[torch.Tensor]], max_norm: float,
                    eps: float = 1e-6) -> torch.Tensor:
    """Scales the gradients of ``parameters`` (or of one tensor) in place to a
    global norm of at most max_norm; returns the norm before (one device
    float32).  Gradients that are not contiguous are scaled in a copy and copied
    back.  A training loop whose gradients keep their buffers builds an
    api.GradList once instead."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    parameters = list(parameters)
    grads = [p.grad for p in parameters if p.grad is not None]
    if not grads:
        return torch.zeros(1, dtype=torch.float32, device=parameters[0].device if parameters else "cuda")
    device = grads[0].device
    norm = torch.empty(1, dtype=torch.float32, device=device)
    ws = torch.empty(api.moe_nvfp4_grad_norm_workspace_bytes(len(grads)), dtype=torch.uint8, device=device)
    strided = [i for i, g in enumerate(grads) if not g.is_contiguous()]
    packed = list(grads)
    for i in strided:
        packed[i] = grads[i].detach().contiguous()
    gl = api.GradList(packed)
    api.moe_nvfp4_grad_norm(gl, norm, ws)
    api.moe_nvfp4_grad_clip(gl, norm, max_norm, eps)
    for i in strided:
        grads[i].detach().copy_(packed[i])
    return norm
