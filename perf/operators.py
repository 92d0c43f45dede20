"""The training operators of a Mixture-of-Experts block, as cases to be timed and compared.

Four operators, each with its gradient:
  rows     routes sorted by expert; token rows copied to their expert's segment (dispatch) and back with the
           router weights (combine)
  experts  every expert's matrix product over its own rows: y = x W^T, dx = dy W, dW = dy^T x (BF16)
  norm     layer norm over the hidden size, with the reduction of the weight's and the bias's gradient
  clip     the global norm of a list of gradients, and the gradients scaled down to a largest norm

`own` false: plain torch operations in 32 bits.  `own` true: this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5          # layer norm
CLIP_EPS = 1e-6     # added to the norm before the division, as gradient clipping commonly does


def listed():
    return [
        # a decoding step of one token at H = 7168, 256 experts, top-8: nothing but latency
        {"name": "rows_forward_token", "op": "rows", "dir": "forward", "T": 1, "H": 7168, "E": 256, "K": 8,
         "dtype": "bf16", "drop": 0.0},
        # a training step's gradient in FP32, an odd hidden size, and routes dropped by a capacity limit
        {"name": "rows_backward_odd_f32", "op": "rows", "dir": "backward", "T": 1023, "H": 1001, "E": 40, "K": 3,
         "dtype": "f32", "drop": 0.1},
        # a prefill of 16384 tokens, both ways
        {"name": "rows_forward_prefill", "op": "rows", "dir": "forward", "T": 16384, "H": 7168, "E": 256, "K": 8,
         "dtype": "bf16", "drop": 0.0},
        {"name": "rows_backward_prefill", "op": "rows", "dir": "backward", "T": 16384, "H": 7168, "E": 256, "K": 8,
         "dtype": "bf16", "drop": 0.02},
        # one token's eight experts at the large shape: the weights' bytes are all that counts
        {"name": "experts_forward_token", "op": "experts", "dir": "forward", "R": 8, "N": 4096, "K": 7168, "E": 16,
         "empty": 0},
        # a small training batch: tens of ragged rows for each of 64 experts, four of them with none
        {"name": "experts_backward_ragged", "op": "experts", "dir": "backward", "R": 2999, "N": 1536, "K": 2048,
         "E": 64, "empty": 4},
        # a compute-bound batch: 1024 rows for each of 16 experts on average, both ways
        {"name": "experts_forward_large", "op": "experts", "dir": "forward", "R": 16384, "N": 4096, "K": 7168, "E": 16,
         "empty": 0},
        {"name": "experts_backward_large", "op": "experts", "dir": "backward", "R": 16384, "N": 4096, "K": 7168,
         "E": 16, "empty": 1},
        # the norm before the layer: a decoding step, and a training batch's gradient
        {"name": "norm_forward_token", "op": "norm", "dir": "forward", "T": 1, "H": 7168, "dtype": "bf16"},
        {"name": "norm_backward_batch", "op": "norm", "dir": "backward", "T": 8191, "H": 7168, "dtype": "bf16"},
        # the gradients of a small layer in FP32, and of a layer of 64 experts in BF16
        {"name": "clip_small_f32", "op": "clip", "H": 250, "I": 128, "E": 8, "dtype": "f32", "max_norm": 1.0},
        {"name": "clip_layer_bf16", "op": "clip", "H": 2048, "I": 768, "E": 64, "dtype": "bf16", "max_norm": 1.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _tokens(rng, hi):
    """A number of rows over the range, odd above 512: no whole number of tiles (the listed cases have those)."""
    n = _log_int(rng, 1, hi - 1)
    return n | 1 if n > 512 else n


def _width(rng, lo, hi, any_number=True):
    """A width over the range: a multiple of 8 three times in four (always, without any_number), else any number;
    none is a multiple of 512 (the listed cases have those)."""
    h = _log_int(rng, lo, hi - 8)
    if not any_number or rng.random() >= 0.25:
        h = h // 8 * 8
    return h + 8 if h % 512 == 0 else h


def draw(rng):
    op = rng.choice(["rows", "experts", "norm", "clip"])
    if op == "rows":
        while True:
            e = _log_int(rng, 2, 256)
            c = {"op": op, "dir": rng.choice(["forward", "backward"]), "T": _tokens(rng, 16384),
                 "H": _width(rng, 64, 7168), "E": e, "K": rng.randint(1, min(8, e)),
                 "dtype": rng.choice(["bf16", "bf16", "f32"]), "drop": rng.choice([0.0, 0.0, 0.05, 0.5])}
            if c["T"] * c["K"] * c["H"] * (4 if c["dtype"] == "f32" else 2) <= 16384 * 8 * 7168 * 2:
                return c
    if op == "experts":
        while True:
            e = _log_int(rng, 1, 64)
            c = {"op": op, "dir": rng.choice(["forward", "backward"]), "R": _tokens(rng, 16384),
                 "N": _width(rng, 64, 7168, False), "K": _width(rng, 64, 7168, False), "E": e,
                 "empty": rng.randint(0, e // 3)}
            if c["R"] * c["N"] * c["K"] <= 16384 * 4096 * 7168 and e * c["N"] * c["K"] <= 16 * 4096 * 7168:
                return c
    if op == "norm":
        return {"op": op, "dir": rng.choice(["forward", "backward"]), "T": _tokens(rng, 8192),
                "H": _width(rng, 64, 7168), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    while True:
        c = {"op": op, "H": _width(rng, 64, 4096), "I": _width(rng, 64, 2048), "E": _log_int(rng, 1, 128),
             "dtype": rng.choice(["bf16", "f32"]), "max_norm": rng.choice([0.5, 1.0, 2.0])}
        if sum(_clip_sizes(c)) * (4 if c["dtype"] == "f32" else 2) <= 64 * 4800000 * 2:
            return c


# ---- inputs -----------------------------------------------------------------------------------------------------

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _clip_sizes(case):
    """The gradients of one layer: norm weight and bias, gate, and each expert's two matrices."""
    h, i, e = case["H"], case["I"], case["E"]
    return [h, h, e * h] + [2 * i * h, h * i] * e


def _counts(case, seed):
    """Rows of each expert: `empty` of them have none, the others a ragged share (one row each if there are no more)."""
    r = torch.Generator().manual_seed(seed)
    e, rows = case["E"], case["R"]
    busy = torch.randperm(e, generator=r)[:e - case["empty"]]
    count = torch.zeros(e, dtype=torch.int64)
    if rows <= len(busy):
        count[busy[:rows]] = 1
    else:
        share = torch.exp(0.4 * torch.randn(len(busy), generator=r))
        more = torch.multinomial(share, rows - len(busy), replacement=True, generator=r)
        count[busy] = 1 + torch.bincount(more, minlength=len(busy))
    return count


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "rows":
        T, H, E, K, dt = case["T"], case["H"], case["E"], case["K"], DTYPES[case["dtype"]]
        # distinct experts for each token, some far more popular than others, weights of a softmax
        score = torch.randn(T, E, generator=gen, device="cuda") + 0.7 * torch.randn(E, generator=gen, device="cuda")
        top, ids = score.topk(K, dim=1)
        if case["drop"]:
            ids = torch.where(torch.rand(T, K, generator=gen, device="cuda") < case["drop"], -1, ids)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["w"] = torch.softmax(top, dim=1).contiguous()
        flat = ids.reshape(-1)
        key = torch.where(flat < 0, E, flat)
        order = torch.argsort(key, stable=True)
        used = int((flat >= 0).sum())
        back = torch.empty_like(order)
        back[order] = torch.arange(T * K, device="cuda")
        s["row_of_route"] = torch.where(flat < 0, -1, back).to(torch.int32).reshape(T, K).contiguous()
        s["route_of_row"] = torch.where(torch.arange(T * K, device="cuda") < used, order, -1).to(torch.int32)
        s["used"] = torch.full((1,), used, dtype=torch.int32, device="cuda")
        s["o_rows"] = _normal(gen, (T * K, H), dt)
        if case["dir"] == "forward":
            s["x"] = _normal(gen, (T, H), dt)
        else:
            s["dy"] = _normal(gen, (T, H), dt)
            s["dx_rows"] = _normal(gen, (T * K, H), dt)
        if own:
            from nvfp4_mixture_experts_router_gb300 import api
            i32 = {"dtype": torch.int32, "device": "cuda"}
            s["out_rows"] = torch.empty(T * K, H, dtype=dt, device="cuda")
            s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
            if case["dir"] == "forward":
                s["order"] = (torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T, K, **i32),
                              torch.empty(T * K, **i32))
                s["ws"] = torch.empty(api.moe_nvfp4_sort_workspace_bytes(T, E, K), dtype=torch.uint8, device="cuda")
            else:
                s["dw"] = torch.empty(T, K, dtype=torch.float32, device="cuda")
    elif case["op"] == "experts":
        R, N, K, E = case["R"], case["N"], case["K"], case["E"]
        count = _counts(case, seed)
        s["most"] = int(count.max())
        s["count"] = count.to(torch.int32).cuda()
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)]).to(torch.int32).cuda()
        s["x"] = _normal(gen, (R, K), torch.bfloat16)
        s["w"] = _normal(gen, (E, N, K), torch.bfloat16, K ** -0.5)
        if case["dir"] == "backward":
            s["dy"] = _normal(gen, (R, N), torch.bfloat16)
        if own:
            bf = {"dtype": torch.bfloat16, "device": "cuda"}
            if case["dir"] == "forward":
                s["out"] = torch.empty(R, N, **bf)
            else:
                s["dx"], s["dw"] = torch.empty(R, K, **bf), torch.empty(E, N, K, **bf)
    elif case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        # a residual stream: an offset and a spread for each channel
        s["x"] = _normal(gen, (T, H), torch.float32) * (0.5 + torch.rand(H, generator=gen, device="cuda"))
        s["x"] = (s["x"] + 0.3 * torch.randn(H, generator=gen, device="cuda")).to(dt)
        s["gamma"] = 1.0 + _normal(gen, (H,), torch.float32, 0.2)
        s["beta"] = _normal(gen, (H,), torch.float32, 0.1)
        if case["dir"] == "backward":
            s["dy"] = _normal(gen, (T, H), dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS)
        if own:
            from nvfp4_mixture_experts_router_gb300 import api
            f32 = {"dtype": torch.float32, "device": "cuda"}
            s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
            if case["dir"] == "forward":
                s["stats"] = (torch.empty(T, **f32), torch.empty(T, **f32))
            else:
                s["dgamma"], s["dbeta"] = torch.empty(H, **f32), torch.empty(H, **f32)
                s["ws"] = torch.empty(api.moe_nvfp4_layer_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    else:
        dt, sizes = DTYPES[case["dtype"]], _clip_sizes(case)
        at, starts = 0, []
        for n in sizes:                       # one buffer, each gradient on a 16-byte boundary, zeros between
            starts.append(at)
            at += -(-n // 8) * 8
        s["flat"] = torch.zeros(at, dtype=dt, device="cuda")
        for a, n in zip(starts, sizes):
            s["flat"][a:a + n] = _normal(gen, (n,), dt, 10.0 ** float(torch.rand((), generator=gen, device="cuda") - 3.0))
        if own:
            from nvfp4_mixture_experts_router_gb300 import api
            s["clipped"] = torch.zeros_like(s["flat"])
            s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
            s["grads"] = api.GradList([s["flat"][a:a + n] for a, n in zip(starts, sizes)],
                                      [s["clipped"][a:a + n] for a, n in zip(starts, sizes)])
            s["ws"] = torch.empty(api.moe_nvfp4_grad_norm_workspace_bytes(len(sizes)), dtype=torch.uint8,
                                  device="cuda")
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    plain = {"rows": _rows_plain, "experts": _experts_plain, "norm": _norm_plain, "clip": _clip_plain}
    kernels = {"rows": _rows_own, "experts": _experts_own, "norm": _norm_own, "clip": _clip_own}
    return (kernels if own else plain)[state["op"]](state)


def _rows_own(s):
    from nvfp4_mixture_experts_router_gb300 import api
    if s["dir"] == "forward":
        count, offsets, row_of_route, route_of_row = s["order"]
        api.moe_nvfp4_sort_routes(s["E"], s["ids"], count, offsets, row_of_route, route_of_row, s["ws"])
        api.moe_nvfp4_dispatch(s["x"], row_of_route, offsets[s["E"]:], s["out_rows"])
        api.moe_nvfp4_combine(s["o_rows"], row_of_route, s["w"], s["out"])
        return {"count": count, "offsets": offsets, "row_of_route": row_of_route, "route_of_row": route_of_row,
                "x_rows": s["out_rows"], "y": s["out"]}
    api.moe_nvfp4_combine_backward(s["dy"], s["o_rows"], s["row_of_route"], s["w"], s["used"], s["out_rows"], s["dw"])
    api.moe_nvfp4_dispatch_backward(s["dx_rows"], s["row_of_route"], s["out"])
    return {"do_rows": s["out_rows"], "dw": s["dw"], "dx": s["out"]}


def _rows_plain(s):
    T, K, E, H = s["T"], s["K"], s["E"], s["H"]
    dt = s["o_rows"].dtype
    places = torch.arange(T * K, device="cuda")
    if s["dir"] == "forward":
        flat = s["ids"].reshape(-1).long()
        kept = (flat >= 0) & (flat < E)
        key = torch.where(kept, flat, E)
        order = torch.argsort(key, stable=True)
        count = torch.zeros(E + 1, dtype=torch.int64, device="cuda").scatter_add_(0, key, torch.ones_like(key))[:E]
        offsets = torch.cat([torch.zeros_like(count[:1]), torch.cumsum(count, 0)])
        filled = places < offsets[E]
        row = torch.where(kept, torch.empty_like(order).scatter_(0, order, places), -1)
        route = torch.where(filled, order, -1)
        x_rows = torch.where(filled[:, None], s["x"].float()[order // K], 0.0)
        weight = torch.where(kept, s["w"].reshape(-1), 0.0)
        part = torch.where(kept[:, None], s["o_rows"].float()[row.clamp(min=0)] * weight[:, None], 0.0)
        return {"count": count.int(), "offsets": offsets.int(), "row_of_route": row.int().view(T, K),
                "route_of_row": route.int(), "x_rows": x_rows.to(dt), "y": part.view(T, K, H).sum(1).to(dt)}
    row = s["row_of_route"].reshape(-1).long()
    route = s["route_of_row"].long()
    kept, filled = row >= 0, route >= 0
    dy = s["dy"].float()
    weight = s["w"].reshape(-1)[route.clamp(min=0)]
    do_rows = torch.where(filled[:, None], weight[:, None] * dy[route.clamp(min=0) // K], 0.0)
    o = s["o_rows"].float()[row.clamp(min=0)].view(T, K, H)
    dw = torch.where(kept.view(T, K), (o * dy[:, None, :]).sum(2), 0.0)
    dx = torch.where(kept[:, None], s["dx_rows"].float()[row.clamp(min=0)], 0.0).view(T, K, H).sum(1)
    return {"do_rows": do_rows.to(dt), "dw": dw, "dx": dx.to(dt)}


def _experts_own(s):
    from nvfp4_mixture_experts_router_gb300 import api
    if s["dir"] == "forward":
        api.moe_nvfp4_expert_linear(s["x"], s["w"], s["count"], s["offsets"], s["out"])
        return {"y": s["out"]}
    api.moe_nvfp4_expert_linear_dgrad(s["dy"], s["w"], s["count"], s["offsets"], s["dx"])
    api.moe_nvfp4_expert_linear_wgrad(s["dy"], s["x"], s["count"], s["offsets"], s["dw"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _experts_plain(s):
    """One batched product over the experts, every expert's rows padded with zeros to the longest segment."""
    R, most = s["R"], s["most"]
    start, count = s["offsets"][:-1].long(), s["count"].long()
    slot = torch.arange(most, device="cuda")
    at = (start[:, None] + slot[None, :]).clamp(max=R - 1)
    there = (slot[None, :] < count[:, None])[:, :, None]
    rows = torch.arange(R, device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].long().contiguous(), rows, right=True)
    home = expert * most + rows - start[expert]
    w = s["w"].float()
    if s["dir"] == "forward":
        x = torch.where(there, s["x"].float()[at], 0.0)
        y = torch.bmm(x, w.transpose(1, 2))
        return {"y": y.reshape(-1, s["N"])[home].to(torch.bfloat16)}
    x = torch.where(there, s["x"].float()[at], 0.0)
    dy = torch.where(there, s["dy"].float()[at], 0.0)
    dx = torch.bmm(dy, w).reshape(-1, s["K"])[home]
    dw = torch.bmm(dy.transpose(1, 2), x)
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


def _norm_own(s):
    from nvfp4_mixture_experts_router_gb300 import api
    if s["dir"] == "forward":
        mean, rstd = s["stats"]
        api.moe_nvfp4_layer_norm(s["x"], s["gamma"], s["beta"], EPS, s["out"], mean, rstd)
        return {"y": s["out"], "mean": mean, "rstd": rstd}
    api.moe_nvfp4_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["out"], s["dgamma"],
                                      s["dbeta"], s["ws"])
    return {"dx": s["out"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def _norm_plain(s):
    x = s["x"].float()
    if s["dir"] == "forward":
        mean = x.mean(1)
        centred = x - mean[:, None]
        rstd = torch.rsqrt((centred * centred).mean(1) + EPS)
        y = centred * rstd[:, None] * s["gamma"] + s["beta"]
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    dy = s["dy"].float()
    hat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"]
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * hat).sum(0), "dbeta": dy.sum(0)}


def _clip_own(s):
    from nvfp4_mixture_experts_router_gb300 import api
    api.moe_nvfp4_grad_norm(s["grads"], s["norm"], s["ws"])
    api.moe_nvfp4_grad_clip(s["grads"], s["norm"], s["max_norm"], CLIP_EPS)
    return {"norm": s["norm"], "grads": s["clipped"]}


def _clip_plain(s):
    g = s["flat"].float()
    norm = (g * g).sum().sqrt().reshape(1)
    scale = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return {"norm": norm, "grads": (g * scale).to(s["flat"].dtype)}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    if case["op"] == "rows":
        T, H, E, K, b = case["T"], case["H"], case["E"], case["K"], 4 if case["dtype"] == "f32" else 2
        rows, kept = T * K, T * K * (1.0 - case["drop"])
        if case["dir"] == "forward":
            return {"bytes": 4 * (2 * rows + 2 * E + 1 + 2 * rows) + b * H * (T + rows + kept + T),
                    "flops": 2.0 * kept * H}
        return {"bytes": 4 * 3 * rows + b * H * (T + kept + rows + kept + T), "flops": 4.0 * kept * H}
    if case["op"] == "experts":
        R, N, K = case["R"], case["N"], case["K"]
        busy = min(R, case["E"] - case["empty"])
        if case["dir"] == "forward":
            return {"bytes": 2 * (R * K + busy * N * K + R * N), "flops": 2.0 * R * N * K}
        return {"bytes": 2 * (R * N + R * K + busy * N * K + R * K + case["E"] * N * K), "flops": 4.0 * R * N * K}
    if case["op"] == "norm":
        T, H, b = case["T"], case["H"], 4 if case["dtype"] == "f32" else 2
        if case["dir"] == "forward":
            return {"bytes": 2 * b * T * H + 8 * H + 8 * T, "flops": 8.0 * T * H}
        return {"bytes": 3 * b * T * H + 12 * H + 8 * T, "flops": 14.0 * T * H}
    n = sum(_clip_sizes(case))
    return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2), "flops": 3.0 * n}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rows":
        T, K, H = s["T"], s["K"], s["H"]
        rows = s["row_of_route"].long()
        if s["dir"] == "forward":
            x_rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
            y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
            for k in range(K):
                t = torch.nonzero(rows[:, k] >= 0).reshape(-1)
                r = rows[t, k]
                x_rows[r] = s["x"][t].double()
                y[t] += s["w"][t, k].double()[:, None] * s["o_rows"][r].double()
            return {"count": None, "offsets": None, "row_of_route": None, "route_of_row": None, "x_rows": x_rows,
                    "y": y}
        do_rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for k in range(K):
            t = torch.nonzero(rows[:, k] >= 0).reshape(-1)
            r = rows[t, k]
            dy = s["dy"][t].double()
            do_rows[r] = s["w"][t, k].double()[:, None] * dy
            dw[t, k] = torch.einsum("th,th->t", dy, s["o_rows"][r].double())
            dx[t] += s["dx_rows"][r].double()
        return {"do_rows": do_rows, "dw": dw, "dx": dx}
    if case["op"] == "experts":
        at = s["offsets"].tolist()
        if s["dir"] == "forward":
            y = torch.zeros(s["R"], s["N"], dtype=torch.float64, device="cuda")
            for e in range(s["E"]):
                y[at[e]:at[e + 1]] = s["x"][at[e]:at[e + 1]].double() @ s["w"][e].double().T
            return {"y": y}
        dx = torch.zeros(s["R"], s["K"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["E"], s["N"], s["K"], dtype=torch.float64, device="cuda")
        for e in range(s["E"]):
            dy = s["dy"][at[e]:at[e + 1]].double()
            dx[at[e]:at[e + 1]] = dy @ s["w"][e].double()
            dw[e] = dy.T @ s["x"][at[e]:at[e + 1]].double()
        return {"dx": dx, "dw": dw}
    if case["op"] == "norm":
        x = s["x"].double()
        if s["dir"] == "forward":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = 1.0 / (var + EPS).sqrt()
            y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) / (var + EPS).sqrt()[:, None],
                              s["gamma"].double())
            return {"y": y, "mean": mean, "rstd": rstd}
        # the gradient of sum(dy * y) by differentiation
        x.requires_grad_(True)
        gamma = s["gamma"].double().requires_grad_(True)
        beta = s["beta"].double().requires_grad_(True)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = (x - mean[:, None]) / (var + EPS).sqrt()[:, None] * gamma + beta
        dx, dgamma, dbeta = torch.autograd.grad((y * s["dy"].double()).sum(), [x, gamma, beta])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    g = s["flat"]
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for part in g.split(1 << 26):
        total += torch.linalg.vector_norm(part.double()) ** 2
    norm = total.sqrt()
    scale = min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
    return {"norm": norm.reshape(1), "grads": g.double() * scale}

