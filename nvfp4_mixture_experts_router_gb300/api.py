"""Python binding of libmoe_nvfp4.so (ctypes).  Argument marshalling only:
every step of the layer runs in the library's CUDA kernels.  PyTorch
supplies device memory and streams.

The functions carry the C names (moe_nvfp4_*); ``MoELayer`` bundles the
buffers of one layer for convenience.  There is no CPU fallback: loading
fails loudly if the library is missing or the device is not sm_103a.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_nvfp4.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_TIMEOUT = range(6)
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT"}

MOE_ACT_SWIGLU = 0
MOE_ACT_RELU2 = 1
MOE_W4A4_PER_TENSOR = 0 << 2
MOE_W4A4_PER_TOKEN = 1 << 2
MOE_W4A16 = 2 << 2
MOE_ROUTER_W_ON_INPUT = 1 << 4
MOE_FINALIZE_DETERMINISTIC = 1 << 5
MOE_ROUTE_NO_RENORM = 1 << 6
MOE_GEMM_PAIRS_NEVER = 1 << 7
MOE_GEMM_PAIRS_ALWAYS = 1 << 8
MOE_QUANT_4OVER6 = 1 << 9
MOE_FUSED_LAYER = 1 << 10
MOE_GEMM_SWAP_NEVER = 1 << 11
MOE_GEMM_SWAP_ALWAYS = 1 << 12
MOE_DEBUG_FC1_SKIP_STAGE = 1 << 13
MOE_ROUTER_GEMM = 1 << 14
MOE_W8A8_MXFP8 = 3 << 2

MOE_DTYPE_BF16, MOE_DTYPE_F32 = 0, 1


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS_NAMES.get(code, code)}")
        self.code = code


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int), ("E", ctypes.c_int),
                ("K", ctypes.c_int)]


_LAYOUT_FIELDS = ["rows_cap", "status", "topk_ids", "topk_w", "count", "offsets", "padded_offsets", "meta",
                  "unit_base", "unit_mask", "row_of_route", "route_of_row", "tile_expert", "tile_pair", "tile_half", "g1",
                  "xq_codes", "xq_sf", "h_f32", "g2", "hq_codes", "hq_sf", "x_bf16_perm", "h_bf16", "o_bf16",
                  "y_acc", "logits", "total"]


class moe_workspace_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in _LAYOUT_FIELDS]


_lib = None


def lib():
    """Load libmoe_nvfp4.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m nvfp4_mixture_experts_router_gb300.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        P, S = ctypes.c_void_p, moe_shape
        u32, i64, sz = ctypes.c_uint32, ctypes.c_int64, ctypes.c_size_t
        c, f = ctypes.c_int, ctypes.c_float
        sig = {
            "moe_nvfp4_version": (ctypes.c_char_p, []),
            "moe_nvfp4_prepared_bytes": (sz, [S, u32]),
            "moe_nvfp4_prepare_weights": (ctypes.c_int, [S, u32, P, P, P, sz, P]),
            "moe_nvfp4_workspace_bytes": (sz, [S, u32]),
            "moe_nvfp4_workspace_layout": (ctypes.c_int, [S, u32, ctypes.POINTER(moe_workspace_layout)]),
            "moe_nvfp4_forward": (ctypes.c_int, [S, u32, P, P, P, P, P, P, P, sz, P, P]),
            "moe_nvfp4_forward_routed": (ctypes.c_int, [S, u32, P, P, P, P, P, P, P, sz, P, P]),
            "moe_nvfp4_forward_staged": (ctypes.c_int, [S, u32, P, P, P, P, P, P, P, sz, P, P,
                                                        ctypes.POINTER(ctypes.c_void_p)]),
            "moe_nvfp4_forward_launches": (ctypes.c_int, [S, u32]),
            "moe_nvfp4_last_device_status": (ctypes.c_int, [P, P]),
            "moe_nvfp4_debug_convert": (ctypes.c_int, [P, i64, P, P, P]),
            "moe_nvfp4_route_noalloc": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, u32, P, P,
                                                       P, P, P, P, P, P, P, P]),
            "moe_nvfp4_router_logits": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, P, P, P, P]),
            "moe_nvfp4_forward_gate": (ctypes.c_int, [S, u32, P, P, P, P, P, P, P, sz, P, P]),
            # training operators (moe_nvfp4_train.h)
            "moe_nvfp4_sort_workspace_bytes": (sz, [c, c, c]),
            "moe_nvfp4_sort_routes": (c, [c, c, c, P, P, P, P, P, P, sz, P]),
            "moe_nvfp4_dispatch": (c, [c, c, c, i64, c, P, i64, P, P, P, P]),
            "moe_nvfp4_dispatch_backward": (c, [c, c, c, i64, c, P, P, P, i64, P]),
            "moe_nvfp4_combine": (c, [c, c, c, i64, c, P, P, P, P, i64, P]),
            "moe_nvfp4_combine_backward": (c, [c, c, c, i64, c, P, i64, P, P, P, P, P, P, P]),
            "moe_nvfp4_expert_linear": (c, [i64, c, c, c, P, P, P, P, P, P, P]),
            "moe_nvfp4_expert_linear_dgrad": (c, [i64, c, c, c, P, P, P, P, P, P, P]),
            "moe_nvfp4_expert_linear_wgrad": (c, [i64, c, c, c, P, P, P, P, P, P, P]),
            "moe_nvfp4_layer_norm": (c, [c, c, c, P, i64, P, P, f, P, i64, P, P, P]),
            "moe_nvfp4_layer_norm_workspace_bytes": (sz, [c, c]),
            "moe_nvfp4_layer_norm_backward": (c, [c, c, c, P, i64, P, i64, P, P, P, P, i64, P, P, P, sz, P]),
            "moe_nvfp4_grad_norm_workspace_bytes": (sz, [c]),
            "moe_nvfp4_grad_norm": (c, [c, P, P, P, P, P, sz, P]),
            "moe_nvfp4_grad_clip": (c, [c, P, P, P, P, P, f, f, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


EXPORTED = ["moe_nvfp4_version", "moe_nvfp4_prepared_bytes", "moe_nvfp4_prepare_weights",
            "moe_nvfp4_workspace_bytes", "moe_nvfp4_workspace_layout", "moe_nvfp4_forward",
            "moe_nvfp4_forward_routed",
            "moe_nvfp4_forward_staged", "moe_nvfp4_forward_launches",
            "moe_nvfp4_last_device_status", "moe_nvfp4_debug_convert", "moe_nvfp4_route_noalloc",
            "moe_nvfp4_router_logits", "moe_nvfp4_forward_gate"]
EXPORTED.sort()
EXPORTED_TRAIN = ["moe_nvfp4_sort_workspace_bytes", "moe_nvfp4_sort_routes", "moe_nvfp4_dispatch",
                  "moe_nvfp4_dispatch_backward", "moe_nvfp4_combine", "moe_nvfp4_combine_backward",
                  "moe_nvfp4_expert_linear", "moe_nvfp4_expert_linear_dgrad", "moe_nvfp4_expert_linear_wgrad",
                  "moe_nvfp4_layer_norm", "moe_nvfp4_layer_norm_workspace_bytes", "moe_nvfp4_layer_norm_backward",
                  "moe_nvfp4_grad_norm_workspace_bytes", "moe_nvfp4_grad_norm", "moe_nvfp4_grad_clip"]
EXPORTED_TRAIN.sort()
NUM_STAGE_EVENTS = 8
STAGES = ["router", "permute", "quantize_x", "fc1", "quantize_h", "fc2", "finalize"]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn: str, code: int):
    if code != MOE_OK:
        raise MoEError(fn, code)


def shape(T: int, H: int, I: int, E: int, K: int) -> moe_shape:
    return moe_shape(T, H, I, E, K)


# ---- C entry points ---------------------------------------------------------

def moe_nvfp4_version() -> str:
    return lib().moe_nvfp4_version().decode()


def moe_nvfp4_prepared_bytes(s: moe_shape, flags: int) -> int:
    return int(lib().moe_nvfp4_prepared_bytes(s, flags))


def moe_nvfp4_workspace_bytes(s: moe_shape, flags: int) -> int:
    return int(lib().moe_nvfp4_workspace_bytes(s, flags))


def moe_nvfp4_workspace_layout(s: moe_shape, flags: int) -> dict:
    out = moe_workspace_layout()
    _check("moe_nvfp4_workspace_layout", lib().moe_nvfp4_workspace_layout(s, flags, ctypes.byref(out)))
    return {n: int(getattr(out, n)) for n in _LAYOUT_FIELDS}


def moe_nvfp4_prepare_weights(s: moe_shape, flags: int, w1_bf16: torch.Tensor, w2_bf16: torch.Tensor,
                              prepared: torch.Tensor, stream=None) -> None:
    code = lib().moe_nvfp4_prepare_weights(s, flags, _ptr(w1_bf16), _ptr(w2_bf16), _ptr(prepared),
                                           prepared.numel() * prepared.element_size(), _stream(stream))
    _check("moe_nvfp4_prepare_weights", code)


def moe_nvfp4_forward(s: moe_shape, flags: int, x_bf16: torch.Tensor, router_logits: torch.Tensor,
                      router_bias: Optional[torch.Tensor], act_scale_fc1: Optional[torch.Tensor],
                      act_scale_fc2: Optional[torch.Tensor], prepared: torch.Tensor, workspace: torch.Tensor,
                      y_bf16: torch.Tensor, stream=None) -> None:
    code = lib().moe_nvfp4_forward(s, flags, _ptr(x_bf16), _ptr(router_logits), _ptr(router_bias),
                                   _ptr(act_scale_fc1), _ptr(act_scale_fc2), _ptr(prepared), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(y_bf16), _stream(stream))
    _check("moe_nvfp4_forward", code)


def moe_nvfp4_forward_routed(s: moe_shape, flags: int, x_bf16: torch.Tensor, topk_ids: torch.Tensor,
                             topk_weights: torch.Tensor, act_scale_fc1: Optional[torch.Tensor],
                             act_scale_fc2: Optional[torch.Tensor], prepared: torch.Tensor, workspace: torch.Tensor,
                             y_bf16: torch.Tensor, stream=None) -> None:
    """Forward on caller-supplied routing: topk_ids int32 [T, K], topk_weights
    float32 [T, K] (CUDA, contiguous)."""
    if topk_ids.dtype != torch.int32 or topk_weights.dtype != torch.float32:
        raise TypeError("topk_ids must be int32 and topk_weights float32")
    if not (topk_ids.is_contiguous() and topk_weights.is_contiguous()):
        raise ValueError("topk_ids and topk_weights must be contiguous")
    if tuple(topk_ids.shape) != (s.T, s.K) or tuple(topk_weights.shape) != (s.T, s.K):
        raise ValueError(f"routing arrays must be [{s.T}, {s.K}]")
    code = lib().moe_nvfp4_forward_routed(s, flags, _ptr(x_bf16), _ptr(topk_ids), _ptr(topk_weights),
                                          _ptr(act_scale_fc1), _ptr(act_scale_fc2), _ptr(prepared),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _ptr(y_bf16), _stream(stream))
    _check("moe_nvfp4_forward_routed", code)


def moe_nvfp4_router_logits(x_bf16: torch.Tensor, gate_w_bf16: torch.Tensor, logits: torch.Tensor,
                            stream=None) -> None:
    """logits [T, E] float32 = x [T, H] . gate_w [E, H]^T (BF16, CUDA, contiguous)."""
    T, H = x_bf16.shape
    E = gate_w_bf16.shape[0]
    if x_bf16.dtype != torch.bfloat16 or gate_w_bf16.dtype != torch.bfloat16 or logits.dtype != torch.float32:
        raise TypeError("x and gate_w must be bfloat16, logits float32")
    if tuple(gate_w_bf16.shape) != (E, H) or tuple(logits.shape) != (T, E):
        raise ValueError("shapes must be x [T, H], gate_w [E, H], logits [T, E]")
    if not (x_bf16.is_contiguous() and gate_w_bf16.is_contiguous() and logits.is_contiguous()):
        raise ValueError("x, gate_w and logits must be contiguous")
    code = lib().moe_nvfp4_router_logits(T, E, H, _ptr(x_bf16), _ptr(gate_w_bf16), _ptr(logits), _stream(stream))
    _check("moe_nvfp4_router_logits", code)


def moe_nvfp4_forward_gate(s: moe_shape, flags: int, x_bf16: torch.Tensor, gate_w_bf16: torch.Tensor,
                           router_bias: Optional[torch.Tensor], act_scale_fc1: Optional[torch.Tensor],
                           act_scale_fc2: Optional[torch.Tensor], prepared: torch.Tensor, workspace: torch.Tensor,
                           y_bf16: torch.Tensor, stream=None) -> None:
    """Forward from the gate projection: flags must include MOE_ROUTER_GEMM;
    gate_w_bf16 is W_g [E, H] (CUDA, contiguous)."""
    if gate_w_bf16.dtype != torch.bfloat16 or tuple(gate_w_bf16.shape) != (s.E, s.H):
        raise ValueError(f"gate_w must be bfloat16 [{s.E}, {s.H}]")
    code = lib().moe_nvfp4_forward_gate(s, flags, _ptr(x_bf16), _ptr(gate_w_bf16), _ptr(router_bias),
                                        _ptr(act_scale_fc1), _ptr(act_scale_fc2), _ptr(prepared), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _ptr(y_bf16), _stream(stream))
    _check("moe_nvfp4_forward_gate", code)


def moe_nvfp4_forward_staged(s: moe_shape, flags: int, x_bf16, router_logits, router_bias, act_scale_fc1,
                             act_scale_fc2, prepared, workspace, y_bf16, events, stream=None) -> None:
    """Forward that records the torch.cuda.Event objects ``events``
    (NUM_STAGE_EVENTS, timing enabled) at the stage boundaries."""
    for ev in events:
        if not ev.cuda_event:       # torch creates the CUDA event lazily, on its first record
            ev.record(stream)
    arr = (ctypes.c_void_p * NUM_STAGE_EVENTS)(*[ctypes.c_void_p(ev.cuda_event) for ev in events])
    code = lib().moe_nvfp4_forward_staged(s, flags, _ptr(x_bf16), _ptr(router_logits), _ptr(router_bias),
                                          _ptr(act_scale_fc1), _ptr(act_scale_fc2), _ptr(prepared),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _ptr(y_bf16), _stream(stream), arr)
    _check("moe_nvfp4_forward_staged", code)


def moe_nvfp4_forward_launches(s: moe_shape, flags: int) -> int:
    return int(lib().moe_nvfp4_forward_launches(s, flags))


def moe_nvfp4_last_device_status(workspace: torch.Tensor, stream=None) -> int:
    return int(lib().moe_nvfp4_last_device_status(_ptr(workspace), _stream(stream)))


def moe_nvfp4_debug_convert(x: torch.Tensor, stream=None):
    """Device E4M3 and E2M1 codes of the float32 CUDA tensor x."""
    x = x.contiguous()
    e4 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    e2 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check("moe_nvfp4_debug_convert",
           lib().moe_nvfp4_debug_convert(_ptr(x), x.numel(), _ptr(e4), _ptr(e2), _stream(stream)))
    return e4, e2


def moe_nvfp4_route_noalloc(T: int, E: int, K: int, flags: int, router_logits: torch.Tensor,
                            router_bias: Optional[torch.Tensor], out: dict, stream=None) -> None:
    """Routing + permutation into the caller's buffers, with the library's
    fixed device scratch instead of a workspace (for callers that cannot
    allocate device memory).  ``out`` holds int32/float32 CUDA tensors
    topk_ids, topk_w, count, offsets, padded_offsets, row_of_route,
    route_of_row (sizes as in include/moe_nvfp4.h)."""
    code = lib().moe_nvfp4_route_noalloc(T, E, K, flags, _ptr(router_logits), _ptr(router_bias),
                                         _ptr(out["topk_ids"]), _ptr(out["topk_w"]), _ptr(out["count"]),
                                         _ptr(out["offsets"]), _ptr(out["padded_offsets"]),
                                         _ptr(out["row_of_route"]), _ptr(out["route_of_row"]), _stream(stream))
    _check("moe_nvfp4_route_noalloc", code)


# ---- training operators (moe_nvfp4_train.h) --------------------------------------

def _handle(stream) -> int:
    """The cudaStream_t of ``stream``, or of the current device's current stream
    (read without building a torch.cuda.Stream: 0.1 us instead of 3)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _rows2d(name: str, t: torch.Tensor, dtype: Optional[torch.dtype] = None) -> tuple:
    """(T, H, row stride in elements) of a CUDA tensor [T, H] with contiguous rows."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [T, H]")
    if (dtype is not None and t.dtype is not dtype) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be {dtype or 'bfloat16 or float32'}")
    T, H = t.shape
    if t.is_contiguous():
        return T, H, H
    if H > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    # the stride of a single row, and of none, says nothing
    return T, H, (t.stride(0) if T > 1 else H)


def _space(workspace: torch.Tensor) -> tuple:
    """Address and size of a workspace."""
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.nbytes


def _flat(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple) -> int:
    """The address of a contiguous CUDA tensor of the given type and shape."""
    if t.dtype is not dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}")
    return t.data_ptr()


_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32}


def moe_nvfp4_sort_workspace_bytes(T: int, E: int, K: int) -> int:
    return int(lib().moe_nvfp4_sort_workspace_bytes(T, E, K))


def moe_nvfp4_sort_routes(E: int, topk_ids: torch.Tensor, count: torch.Tensor, offsets: torch.Tensor,
                          row_of_route: torch.Tensor, route_of_row: torch.Tensor, workspace: torch.Tensor,
                          stream=None) -> None:
    """Routes of topk_ids [T, K] sorted by expert (stable; ids outside [0, E)
    are dropped): count [E], offsets [E + 1], row_of_route [T, K] and
    route_of_row [T * K], all int32."""
    T, K = topk_ids.shape
    i32 = torch.int32
    code = lib().moe_nvfp4_sort_routes(
        T, E, K, _flat("topk_ids", topk_ids, i32, (T, K)), _flat("count", count, i32, (E,)),
        _flat("offsets", offsets, i32, (E + 1,)), _flat("row_of_route", row_of_route, i32, (T, K)),
        _flat("route_of_row", route_of_row, i32, (T * K,)), *_space(workspace), _handle(stream))
    _check("moe_nvfp4_sort_routes", code)


def _row_args(what: str, tokens: torch.Tensor, rows: torch.Tensor, row_of_route: torch.Tensor) -> tuple:
    """Checks token rows [T, H], expert-ordered rows [rows, H] of the same type
    and row_of_route [T, K]; returns (T, H, K, rows, dtype), the tokens' row
    stride and row_of_route's address."""
    T, H, stride = _rows2d(what, tokens)
    if rows.dim() != 2 or rows.dtype is not tokens.dtype or not rows.is_cuda or rows.shape[1] != H \
            or not rows.is_contiguous():
        raise ValueError(f"the expert-ordered rows must be contiguous [rows, {H}] of {tokens.dtype}")
    K = row_of_route.shape[-1]
    return (T, H, K, rows.shape[0], _DTYPES[tokens.dtype]), stride, \
        _flat("row_of_route", row_of_route, torch.int32, (T, K))


def _scalar_i32(name: str, t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.dtype is not torch.int32 or not t.is_cuda or t.numel() != 1:
        raise ValueError(f"{name} must be one CUDA int32")
    return t.data_ptr()


def moe_nvfp4_dispatch(x: torch.Tensor, row_of_route: torch.Tensor, rows_used: Optional[torch.Tensor],
                       x_rows: torch.Tensor, stream=None) -> None:
    """x_rows[row_of_route[t, k]] = x[t]; rows from rows_used (one device int32,
    None: none) on are set to zero."""
    sizes, stride, ror = _row_args("x", x, x_rows, row_of_route)
    code = lib().moe_nvfp4_dispatch(*sizes, x.data_ptr(), stride, ror, _scalar_i32("rows_used", rows_used),
                                    x_rows.data_ptr(), _handle(stream))
    _check("moe_nvfp4_dispatch", code)


def moe_nvfp4_dispatch_backward(dx_rows: torch.Tensor, row_of_route: torch.Tensor, dx: torch.Tensor,
                                stream=None) -> None:
    """dx[t] = sum_k dx_rows[row_of_route[t, k]]."""
    sizes, stride, ror = _row_args("dx", dx, dx_rows, row_of_route)
    code = lib().moe_nvfp4_dispatch_backward(*sizes, dx_rows.data_ptr(), ror, dx.data_ptr(), stride, _handle(stream))
    _check("moe_nvfp4_dispatch_backward", code)


def moe_nvfp4_combine(o_rows: torch.Tensor, row_of_route: torch.Tensor, topk_w: torch.Tensor, y: torch.Tensor,
                      stream=None) -> None:
    """y[t] = sum_k topk_w[t, k] * o_rows[row_of_route[t, k]]."""
    sizes, stride, ror = _row_args("y", y, o_rows, row_of_route)
    w = _flat("topk_w", topk_w, torch.float32, (sizes[0], sizes[2]))
    code = lib().moe_nvfp4_combine(*sizes, o_rows.data_ptr(), ror, w, y.data_ptr(), stride, _handle(stream))
    _check("moe_nvfp4_combine", code)


def moe_nvfp4_combine_backward(dy: torch.Tensor, o_rows: torch.Tensor, row_of_route: torch.Tensor,
                               topk_w: torch.Tensor, rows_used: Optional[torch.Tensor], do_rows: torch.Tensor,
                               dw: torch.Tensor, stream=None) -> None:
    """do_rows[row_of_route[t, k]] = topk_w[t, k] * dy[t] (rows from rows_used on
    set to zero) and dw[t, k] = <dy[t], o_rows[row_of_route[t, k]]>."""
    sizes, stride, ror = _row_args("dy", dy, o_rows, row_of_route)
    T, H, K, rows, _ = sizes
    code = lib().moe_nvfp4_combine_backward(
        *sizes, dy.data_ptr(), stride, o_rows.data_ptr(), ror, _flat("topk_w", topk_w, torch.float32, (T, K)),
        _scalar_i32("rows_used", rows_used), _flat("do_rows", do_rows, dy.dtype, (rows, H)),
        _flat("dw", dw, torch.float32, (T, K)), _handle(stream))
    _check("moe_nvfp4_combine_backward", code)


def _expert_product(fn: str, sizes: tuple, a: torch.Tensor, a_shape: tuple, b: torch.Tensor, b_shape: tuple,
                    count: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor, out_shape: tuple,
                    status: Optional[torch.Tensor], stream) -> None:
    bf16, E = torch.bfloat16, sizes[3]
    if offsets.dtype is not torch.int32 or not offsets.is_cuda:
        raise TypeError("offsets must be CUDA int32")
    if offsets.dim() != 1 or offsets.shape[0] < E or not offsets.is_contiguous():
        raise ValueError(f"offsets must be contiguous [{E}] or longer")
    if status is not None and (status.element_size() != 4 or not status.is_cuda or status.numel() != 1):
        raise ValueError("status must be one CUDA 32-bit integer")
    code = getattr(lib(), fn)(*sizes, _flat("the first operand", a, bf16, a_shape),
                              _flat("the second operand", b, bf16, b_shape), _flat("count", count, torch.int32, (E,)),
                              offsets.data_ptr(), _flat("the output", out, bf16, out_shape),
                              None if status is None else status.data_ptr(), _handle(stream))
    _check(fn, code)


def moe_nvfp4_expert_linear(x_rows: torch.Tensor, w: torch.Tensor, count: torch.Tensor, offsets: torch.Tensor,
                            y_rows: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """y_rows[r] = x_rows[r] w[e]^T for the rows [offsets[e], offsets[e] + count[e])
    of every expert e: x_rows [rows, K], w [E, N, K], y_rows [rows, N], BF16."""
    E, N, K = w.shape
    R = x_rows.shape[0]
    _expert_product("moe_nvfp4_expert_linear", (R, N, K, E), x_rows, (R, K), w, (E, N, K), count, offsets, y_rows,
                    (R, N), status, stream)


def moe_nvfp4_expert_linear_dgrad(dy_rows: torch.Tensor, w: torch.Tensor, count: torch.Tensor, offsets: torch.Tensor,
                                  dx_rows: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx_rows[r] = dy_rows[r] w[e]: dy_rows [rows, N], w [E, N, K], dx_rows [rows, K], BF16."""
    E, N, K = w.shape
    R = dy_rows.shape[0]
    _expert_product("moe_nvfp4_expert_linear_dgrad", (R, N, K, E), dy_rows, (R, N), w, (E, N, K), count, offsets,
                    dx_rows, (R, K), status, stream)


def moe_nvfp4_expert_linear_wgrad(dy_rows: torch.Tensor, x_rows: torch.Tensor, count: torch.Tensor,
                                  offsets: torch.Tensor, dw: torch.Tensor, status: Optional[torch.Tensor] = None,
                                  stream=None) -> None:
    """dw[e] = sum over expert e's rows r of dy_rows[r]^T x_rows[r]: dw [E, N, K], BF16."""
    E, N, K = dw.shape
    R = dy_rows.shape[0]
    _expert_product("moe_nvfp4_expert_linear_wgrad", (R, N, K, E), dy_rows, (R, N), x_rows, (R, K), count, offsets, dw,
                    (E, N, K), status, stream)


def moe_nvfp4_layer_norm(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], eps: float,
                         y: torch.Tensor, mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """y = (x - mean) * rstd * gamma + beta over the rows of x [T, H]; gamma, beta
    [H], mean and rstd [T] float32 (mean and rstd may both be None)."""
    T, H, xs = _rows2d("x", x)
    ys = _rows2d("y", y, x.dtype)[2]
    if y.shape != x.shape:
        raise ValueError("y must have the shape of x")
    f32 = torch.float32
    code = lib().moe_nvfp4_layer_norm(
        T, H, _DTYPES[x.dtype], x.data_ptr(), xs, _flat("gamma", gamma, f32, (H,)),
        None if beta is None else _flat("beta", beta, f32, (H,)), eps, y.data_ptr(), ys,
        None if mean is None else _flat("mean", mean, f32, (T,)),
        None if rstd is None else _flat("rstd", rstd, f32, (T,)), _handle(stream))
    _check("moe_nvfp4_layer_norm", code)


def moe_nvfp4_layer_norm_workspace_bytes(T: int, H: int) -> int:
    return int(lib().moe_nvfp4_layer_norm_workspace_bytes(T, H))


def moe_nvfp4_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor,
                                  rstd: torch.Tensor, dx: torch.Tensor, dgamma: torch.Tensor,
                                  dbeta: Optional[torch.Tensor], workspace: torch.Tensor, stream=None) -> None:
    """dx [T, H], dgamma and dbeta [H] of the layer norm with the forward's mean and rstd [T]."""
    T, H, xs = _rows2d("x", x)
    dys, dxs = _rows2d("dy", dy, x.dtype)[2], _rows2d("dx", dx, x.dtype)[2]
    if dy.shape != x.shape or dx.shape != x.shape:
        raise ValueError("dy and dx must have the shape of x")
    f32 = torch.float32
    code = lib().moe_nvfp4_layer_norm_backward(
        T, H, _DTYPES[x.dtype], dy.data_ptr(), dys, x.data_ptr(), xs, _flat("gamma", gamma, f32, (H,)),
        _flat("mean", mean, f32, (T,)), _flat("rstd", rstd, f32, (T,)), dx.data_ptr(), dxs,
        _flat("dgamma", dgamma, f32, (H,)), None if dbeta is None else _flat("dbeta", dbeta, f32, (H,)),
        *_space(workspace), _handle(stream))
    _check("moe_nvfp4_layer_norm_backward", code)


class GradList:
    """A list of gradients (contiguous CUDA tensors, bfloat16 or float32) and
    where their clipped values go (``out``; the gradients themselves without
    it).  Built once for buffers that stay where they are; it holds the tensors
    and their addresses."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError("as many outputs as gradients")
        for g, o in zip(self.grads, self.out):
            if g.dtype not in _DTYPES or o.dtype != g.dtype or not (g.is_cuda and o.is_cuda):
                raise TypeError("gradients must be bfloat16 or float32 CUDA tensors, each output of its gradient's type")
            if o.numel() != g.numel() or not (g.is_contiguous() and o.is_contiguous()):
                raise ValueError("gradients and outputs must be contiguous and of the same size")
        n = self.n = len(self.grads)
        self.c_grads = (ctypes.c_void_p * n)(*[g.data_ptr() for g in self.grads])
        self.c_out = (ctypes.c_void_p * n)(*[o.data_ptr() for o in self.out])
        self.c_numels = (ctypes.c_int64 * n)(*[g.numel() for g in self.grads])
        self.c_dtypes = (ctypes.c_int32 * n)(*[_DTYPES[g.dtype] for g in self.grads])


def moe_nvfp4_grad_norm_workspace_bytes(n: int) -> int:
    return int(lib().moe_nvfp4_grad_norm_workspace_bytes(n))


def moe_nvfp4_grad_norm(grads: GradList, norm: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """norm[0] (float32) = sqrt of the sum of the squares of every gradient's elements."""
    code = lib().moe_nvfp4_grad_norm(grads.n, grads.c_grads, grads.c_numels, grads.c_dtypes,
                                     _flat("norm", norm, torch.float32, (1,)), *_space(workspace),
                                     _handle(stream))
    _check("moe_nvfp4_grad_norm", code)


def moe_nvfp4_grad_clip(grads: GradList, norm: torch.Tensor, max_norm: float, eps: float = 1e-6,
                        stream=None) -> None:
    """out = gradient * min(1, max_norm / (norm + eps)) for every gradient of the list."""
    code = lib().moe_nvfp4_grad_clip(grads.n, grads.c_grads, grads.c_out, grads.c_numels, grads.c_dtypes,
                                     _flat("norm", norm, torch.float32, (1,)), max_norm, eps, _handle(stream))
    _check("moe_nvfp4_grad_clip", code)


# ---- convenience ---------------------------------------------------------------

@dataclass
class MoELayer:
    """Buffers of one MoE layer on one device: prepared weights + workspace."""
    T: int
    H: int
    I: int
    E: int
    K: int
    flags: int
    prepared: torch.Tensor
    workspace: torch.Tensor

    @property
    def shape(self) -> moe_shape:
        return moe_shape(self.T, self.H, self.I, self.E, self.K)

    @classmethod
    def create(cls, T, H, I, E, K, flags, device="cuda") -> "MoELayer":
        s = moe_shape(T, H, I, E, K)
        pb = moe_nvfp4_prepared_bytes(s, flags)
        wb = moe_nvfp4_workspace_bytes(s, flags)
        if pb == 0 or wb == 0:
            raise MoEError("moe_nvfp4_*_bytes", MOE_ERR_INVALID_ARG)
        prepared = torch.empty(pb, dtype=torch.uint8, device=device)
        workspace = torch.empty(wb, dtype=torch.uint8, device=device)
        return cls(T, H, I, E, K, flags, prepared, workspace)

    def prepare(self, w1_bf16: torch.Tensor, w2_bf16: torch.Tensor, stream=None):
        moe_nvfp4_prepare_weights(self.shape, self.flags, w1_bf16, w2_bf16, self.prepared, stream)

    def forward(self, x_bf16, logits, bias=None, g1=None, g2=None, y=None, stream=None) -> torch.Tensor:
        if y is None:
            y = torch.empty(self.T, self.H, dtype=torch.bfloat16, device=x_bf16.device)
        moe_nvfp4_forward(self.shape, self.flags, x_bf16, logits, bias, g1, g2, self.prepared, self.workspace,
                          y, stream)
        return y

    def forward_gate(self, x_bf16, gate_w_bf16, bias=None, g1=None, g2=None, y=None, stream=None) -> torch.Tensor:
        if y is None:
            y = torch.empty(self.T, self.H, dtype=torch.bfloat16, device=x_bf16.device)
        moe_nvfp4_forward_gate(self.shape, self.flags, x_bf16, gate_w_bf16, bias, g1, g2, self.prepared,
                               self.workspace, y, stream)
        return y

    def forward_routed(self, x_bf16, topk_ids, topk_weights, g1=None, g2=None, y=None, stream=None) -> torch.Tensor:
        if y is None:
            y = torch.empty(self.T, self.H, dtype=torch.bfloat16, device=x_bf16.device)
        moe_nvfp4_forward_routed(self.shape, self.flags, x_bf16, topk_ids, topk_weights, g1, g2, self.prepared,
                                 self.workspace, y, stream)
        return y

    # -- views of the intermediates (tests / debugging) --
    def layout(self) -> dict:
        return moe_nvfp4_workspace_layout(self.shape, self.flags)

    def view(self, name: str, dtype: torch.dtype, numel: int) -> torch.Tensor:
        off = self.layout()[name]
        if off == 2 ** 64 - 1:
            raise KeyError(f"workspace region {name} is not used in this mode")
        nbytes = numel * torch.empty((), dtype=dtype).element_size()
        return self.workspace[off:off + nbytes].view(dtype)

    def prepared_regions(self) -> dict:
        """Byte offsets of the prepared-weight regions (same rule as the library)."""
        def up(v):
            return (v + 255) // 256 * 256
        N1 = 2 * self.I if (self.flags & 3) == MOE_ACT_SWIGLU else self.I
        E, H, I = self.E, self.H, self.I
        mx = (self.flags & (3 << 2)) == MOE_W8A8_MXFP8
        cd, sd = (1, 32) if mx else (2, 16)        # MXFP8: a byte per element, a scale per 32
        o = 0
        r = {}
        for name, nbytes in [("gw1", 4 * E), ("gw2", 4 * E), ("w1_codes", E * N1 * H // cd),
                             ("w1_sf", E * N1 * H // sd), ("w2_codes", E * H * I // cd), ("w2_sf", E * H * I // sd)]:
            r[name] = (o, nbytes)
            o = up(o + nbytes)
        r["total"] = (o, 0)
        return r
