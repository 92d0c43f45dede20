"""The training operators as differentiable torch functions.

Each function allocates its outputs and workspaces with torch, runs on the
current stream, and has its gradient from the same library (api.py has the
calls themselves, on the caller's buffers).  A pre-norm Mixture-of-Experts
block, with the gate's product and the activation in torch:

    y, h = train.rms_norm(x, gamma, residual)           # or train.layer_norm(x, gamma, beta)
    ids, w = train.route(gate(y), K, bias, api.RouteRule(...))      # [T, K]
    routes = train.sort_routes(ids, E)
    z = train.expert_linear(train.dispatch(y, routes), w1, routes)
    o = train.expert_linear(activation(z), w2, routes)
    x = train.combine(o, routes, w)                     # the next block's x, with h as its residual

and its optimizer:

    opt = train.AdamW(parameters, lr=1e-3, state_bits=8)
    opt.step(norm=train.grad_norm(parameters), max_norm=1.0)

examples/moe_block.py trains one such block, examples/moe_stack.py a stack of them.
"""
from __future__ import annotations

from dataclasses import dataclass
from functools import cached_property
from typing import Iterable, Optional, Tuple, Union

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


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, K, bias, rule):
        T = logits.shape[0]
        ids = torch.empty(T, K, dtype=torch.int32, device=logits.device)
        w = torch.empty(T, K, dtype=torch.float32, device=logits.device)
        api.moe_nvfp4_route_topk(logits, bias, rule, ids, w)
        ctx.rule = rule
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        logits, ids = ctx.saved_tensors
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        api.moe_nvfp4_route_topk_backward(logits, ids, dw.contiguous(), ctx.rule, dlogits)
        return dlogits, None, None, None


def route(logits: torch.Tensor, K: int, bias: Optional[torch.Tensor] = None,
          rule: api.RouteRule = api.RouteRule()) -> Tuple[torch.Tensor, torch.Tensor]:
    """The K experts of each token and their weights, [T, K] int32 and FP32, from
    logits [T, E] (BF16 or FP32).  The bias [E] FP32 enters the choice alone and has
    no gradient: a training loop moves it against the experts' load (Routes.count)."""
    return _Route.apply(logits, K, None if bias is None else bias.detach(), rule)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, eps):
        new = lambda: torch.empty(x.shape, dtype=x.dtype, device=x.device)      # noqa: E731
        y, h = new(), None if residual is None else new()
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        api.moe_nvfp4_rms_norm(x, residual, gamma, eps, h, y, None, None, rstd)
        ctx.save_for_backward(x if h is None else h, gamma, rstd)
        ctx.with_residual = h is not None
        ctx.set_materialize_grads(False)
        return y if h is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, gamma, rstd = ctx.saved_tensors
        if dy is None:      # only h was used
            return dh, dh if ctx.with_residual else None, None, None
        dx = torch.empty(h.shape, dtype=h.dtype, device=h.device)
        dgamma = torch.empty_like(gamma)
        ws = torch.empty(api.moe_nvfp4_rms_norm_workspace_bytes(*h.shape), dtype=torch.uint8, device=h.device)
        api.moe_nvfp4_rms_norm_backward(dy.contiguous(), None if dh is None else dh.contiguous(), h, gamma, rstd, dx,
                                        dgamma, ws)
        return dx, dx if ctx.with_residual else None, dgamma, None


def rms_norm(x: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """RMS norm of h = x + residual, [T, H] (BF16 or FP32, both of one type), gamma [H]
    FP32.  Returns y and h, or y alone without a residual (h is x then)."""
    return _RmsNorm.apply(x, residual, gamma, eps)


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


def grad_norm(parameters: Union[torch.Tensor, Iterable[torch.Tensor]]) -> torch.Tensor:
    """The global norm of the gradients of ``parameters`` (one device float32), for
    AdamW.step, which clips on its way; the gradients stay as they are."""
    grads = [p.grad for p in ([parameters] if isinstance(parameters, torch.Tensor) else parameters)
             if p.grad is not None]
    device = grads[0].device if grads else "cuda"
    norm = torch.empty(1, dtype=torch.float32, device=device)
    ws = torch.empty(api.moe_nvfp4_grad_norm_workspace_bytes(len(grads)), dtype=torch.uint8, device=device)
    api.moe_nvfp4_grad_norm(api.GradList([g.detach().contiguous() for g in grads]), norm, ws)
    return norm


_LISTS_KEPT = 8     # of AdamW; those of one step where they are more


class AdamW:
    """AdamW over parameters (BF16 or FP32, contiguous, on one device), a launch for
    each kind of states and 384 tensors (moe_nvfp4_adamw).

    state_bits 8 keeps both moments in E4M3 with a scale for each 256 elements, of
    tensors from min_8bit elements on; master keeps FP32 values of BF16
    parameters, from which these are rounded.  Parameters that changed since their
    last step (a checkpoint loaded, weights swapped in) are read again, as autograd's
    count of changes or their address tells; after a change that neither tells of
    (through .data, or before the replay of a captured step) call read_parameters.
    Parameters without a gradient are left as they are, and count their steps by
    themselves (a launch for each number).
    lr, betas, eps and weight_decay may be set between steps, by a schedule for one;
    parameters that take other ones have an optimizer of their own.
    capturable: the learning rate and the number of the step are read on the device
    (self.lr_step), so that a step captured into a CUDA graph counts on when it is
    replayed; run one step before the capture.  A replay takes its rate from
    lr_step[0]; a step outside of one writes self.lr there where that changed.  All
    parameters then have a gradient in every step, or never."""

    def __init__(self, params: Iterable[torch.Tensor], lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: float = 0.01, state_bits: int = 32, master: bool = True,
                 min_8bit: int = 4096, capturable: bool = False):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.params = list(params)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.steps = [0] * len(self.params)     # of each parameter
        self.state = []
        for p in self.params:
            n, s, dev = p.numel(), {}, dict(device=p.device)
            small = state_bits == 32 or n < min_8bit
            for name in ("exp_avg", "exp_avg_sq"):
                if small:
                    s[name] = torch.zeros(n, dtype=torch.float32, **dev)
                else:
                    s[name] = torch.zeros(n, dtype=torch.uint8, **dev).view(torch.float8_e4m3fn)
                    s[name + "_scale"] = torch.zeros(-(-n // api.MOE_ADAMW_BLOCK), dtype=torch.float32, **dev)
            if master and p.dtype == torch.bfloat16:
                s["master"] = p.detach().float().reshape(-1)
            self.state.append(s)
        # autograd's count of changes, and the address, of the values that the masters are of
        # (None: tensors of inference mode, whose changes are not counted)
        self._seen = [None if p.is_inference() else (p._version, p.data_ptr()) for p in self.params]
        self._masters = any("master" in s for s in self.state)
        self.lr_step = None
        if capturable and self.params:
            self.lr_step = torch.tensor([lr, 0.0], dtype=torch.float32, device=self.params[0].device)
            self._device_lr = lr
        self._lists = {}        # parameters of a launch -> their addresses and the list, the last used behind

    def zero_grad(self, set_to_none: bool = True) -> None:
        for p in self.params:
            if set_to_none or p.grad is None:
                p.grad = None
            else:
                p.grad.zero_()

    @torch.no_grad()
    def _read(self, i: int) -> None:
        """Parameter i into its master: where the two agree, the master's digits stay."""
        p, w = self.params[i], self.state[i].get("master")
        if w is not None:
            q = p.detach().reshape(-1)
            w.copy_(torch.where(w.to(q.dtype) == q, w, q.float()))
        if self._seen[i] is not None:
            self._seen[i] = p._version, p.data_ptr()

    def read_parameters(self) -> None:
        """Takes the parameters as they are for the next step, however they were changed."""
        for i in range(len(self.params)):
            self._read(i)

    @torch.no_grad()
    def step(self, norm: Optional[torch.Tensor] = None, max_norm: float = 1.0, clip_eps: float = 1e-6) -> None:
        """One step.  norm: the gradients' global norm (grad_norm; float32 [1]), by which
        they are clipped to max_norm on the way."""
        groups = {}
        for i, p in enumerate(self.params):
            if p.grad is not None:
                groups.setdefault(self.steps[i], []).append(i)
        if self.lr_step is not None and groups:
            if any(self.steps) and [bool(n) for n in self.steps] != [p.grad is not None for p in self.params]:
                raise ValueError("a capturable AdamW's parameters have a gradient in every step, or never")
            if self._device_lr != self.lr:
                if torch.cuda.is_current_stream_capturing():
                    raise ValueError("the learning rate changed since the last step: run one before the capture")
                self.lr_step[0].fill_(self.lr)
                self._device_lr = self.lr
        rule = api.AdamWRule(self.lr, *self.betas, self.eps, self.weight_decay, max_norm, clip_eps)
        for steps, used in groups.items():
            params = [self.params[i] for i in used]
            at = [p.data_ptr() for p in params]
            grads = [p.grad.contiguous() for p in params]
            if self._masters:
                for i, p, a in zip(used, params, at):
                    if self._seen[i] is not None and self._seen[i] != (p._version, a):
                        self._read(i)
            kept = self._lists.pop(tuple(used), None)
            if kept is None or kept[0] != at:
                get = lambda name: [self.state[i].get(name) for i in used]      # noqa: E731, B023
                kept = at, api.AdamWList(params, grads, get("exp_avg"), get("exp_avg_sq"),
                                         get("exp_avg_scale"), get("exp_avg_sq_scale"), get("master"))
            else:
                kept[1].set_grads(grads)
            self._lists[tuple(used)] = kept
            if self.lr_step is not None:
                self.lr_step[1].add_(1.0)
            try:
                api.moe_nvfp4_adamw(kept[1], rule, steps + 1, norm, self.lr_step)
            except Exception:
                if self.lr_step is not None:
                    self.lr_step[1].sub_(1.0)       # a refused step does not count
                raise
            kept[1].grads = []       # the gradients may go
            torch.autograd.graph.increment_version(params)      # graphs that saved them raise
            for i in used:
                self.steps[i] += 1
            if self._masters:
                for i, p, a in zip(used, params, at):
                    if self._seen[i] is not None:
                        self._seen[i] = p._version, a
        while len(self._lists) > max(_LISTS_KEPT, len(groups)):     # sets of parameters that may not come back
            del self._lists[next(iter(self._lists))]

    def state_dict(self) -> dict:
        steps = list(self.steps)
        if self.lr_step is not None:        # replays count on the device alone
            steps = [int(self.lr_step[1]) if n else 0 for n in steps]
        return {"steps": steps, "state": self.state}

    def load_state_dict(self, saved: dict) -> None:
        """Copies the states of an optimizer of the same parameters and kind."""
        if [{k: (v.shape, v.dtype) for k, v in s.items()} for s in saved["state"]] != \
                [{k: (v.shape, v.dtype) for k, v in s.items()} for s in self.state]:
            raise ValueError("the states are of other parameters, or of another kind")
        if self.lr_step is not None and len(set(saved["steps"]) - {0}) > 1:
            raise ValueError("a capturable AdamW's parameters have the same number of steps")
        for mine, theirs in zip(self.state, saved["state"]):
            for k, v in theirs.items():
                mine[k].copy_(v)
        self.steps = list(saved["steps"])
        if self.lr_step is not None:
            self.lr_step[1].fill_(max(self.steps, default=0))


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
    torch.autograd.graph.increment_version(grads)       # graphs that saved them raise
    for i in strided:
        grads[i].detach().copy_(packed[i])
    return norm
