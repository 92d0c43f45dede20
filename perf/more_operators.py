"""Routing, root-mean-square norm and AdamW, the operators around a Mixture-of-Experts block, as cases to be timed and
compared.

  route    experts chosen from logits: softmax or sigmoid scores, a bias that only chooses, groups of experts, top-k,
           renormalised weights; and the gradient of the logits
  rms      the residual's addition and root-mean-square norm, with the result in the rows' type or in E4M3 with scales;
           and its gradient
  adamw    one AdamW step over a list of tensors: gradients clipped on the way, BF16 or FP32 parameters, FP32 master
           values, states in FP32 or in E4M3

`own` false: plain torch operations in 32 bits (the choice of experts in 64: whole numbers have to be equal).
`own` true: this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0              # largest E4M3 value
LARGEST = 3.4028234663852886e38     # of FP32
RMS_EPS = 1e-6
CLIP_EPS = 1e-6             # added to the norm before the division
STATE_BLOCK = 256           # elements that share a scale in states of 8 bits
STATE_FLUSH = 2.0 ** -100   # a block of states whose largest magnitude is below this is stored as zeros
ADAMW = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "max_norm": 1.0}


def listed():
    return [
        # a decoding step of one token: 256 experts in 8 groups of which 4 are taken, sigmoid scores and a bias
        {"name": "route_forward_token", "op": "route", "dir": "forward", "T": 1, "E": 256, "K": 8, "dtype": "f32",
         "score": "sigmoid", "bias": 0.05, "groups": 8, "top_groups": 4, "pair": True, "renorm": True, "scale": 2.5,
         "masked": 0.0},
        # a middle batch with softmax over 64 experts, top-6, logits straight from a BF16 product (equal ones occur)
        {"name": "route_forward_batch_bf16", "op": "route", "dir": "forward", "T": 511, "E": 64, "K": 6, "dtype": "bf16",
         "score": "softmax", "bias": 0.0, "groups": 1, "top_groups": 1, "pair": False, "renorm": True, "scale": 1.0,
         "masked": 0.0},
        # a prefill of 16384 tokens
        {"name": "route_forward_prefill", "op": "route", "dir": "forward", "T": 16384, "E": 256, "K": 8, "dtype": "f32",
         "score": "sigmoid", "bias": 0.05, "groups": 8, "top_groups": 4, "pair": True, "renorm": True, "scale": 2.5,
         "masked": 0.0},
        # its gradient, and one of weights that are not renormalised (every expert's logit gets some), some experts off
        {"name": "route_backward_prefill", "op": "route", "dir": "backward", "T": 16384, "E": 256, "K": 8, "dtype": "f32",
         "score": "sigmoid", "bias": 0.05, "groups": 8, "top_groups": 4, "pair": True, "renorm": True, "scale": 2.5,
         "masked": 0.0},
        {"name": "route_backward_odd_bf16", "op": "route", "dir": "backward", "T": 4097, "E": 40, "K": 3, "dtype": "bf16",
         "score": "softmax", "bias": 0.0, "groups": 1, "top_groups": 1, "pair": False, "renorm": False, "scale": 1.0,
         "masked": 0.1},
        # a decoding step's norm: residual added, E4M3 with a scale for the row
        {"name": "rms_forward_token_e4m3", "op": "rms", "dir": "forward", "T": 1, "H": 7168, "dtype": "bf16",
         "residual": True, "out": "row"},
        # a prefill's: E4M3 with a power of two for each 32 elements, the sum kept for the next layer
        {"name": "rms_forward_prefill_mx", "op": "rms", "dir": "forward", "T": 16384, "H": 7168, "dtype": "bf16",
         "residual": True, "out": "mx"},
        # a training step in FP32 at an odd width, without a residual
        {"name": "rms_forward_odd_f32", "op": "rms", "dir": "forward", "T": 1023, "H": 1001, "dtype": "f32",
         "residual": False, "out": "same"},
        # a training batch's gradient, the residual stream's own added
        {"name": "rms_backward_batch", "op": "rms", "dir": "backward", "T": 8191, "H": 7168, "dtype": "bf16",
         "residual": True},
        # a small layer in FP32
        {"name": "adamw_small_f32", "op": "adamw", "H": 250, "I": 128, "E": 8, "dtype": "f32", "master": False, "bits": 32},
        # a layer of 64 experts: BF16 with FP32 master values and states, and with states of 8 bits
        {"name": "adamw_layer_master", "op": "adamw", "H": 2048, "I": 768, "E": 64, "dtype": "bf16", "master": True,
         "bits": 32},
        {"name": "adamw_layer_8bit", "op": "adamw", "H": 2048, "I": 768, "E": 64, "dtype": "bf16", "master": False,
         "bits": 8},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "rms", "adamw"])
    if op == "route":
        T = _log_int(rng, 2, 16383)
        groups = rng.choice([1, 1, 2, 4, 5, 8])
        E = max(groups * 2, _log_int(rng, 4, 256) // groups * groups)
        top = rng.randint(max(1, groups // 3), groups)
        return {"op": op, "dir": rng.choice(["forward", "forward", "backward"]), "T": T | 1 if T > 512 else T, "E": E,
                "K": rng.randint(1, min(8, top * (E // groups))), "dtype": rng.choice(["f32", "f32", "bf16"]),
                "score": rng.choice(["softmax", "sigmoid", "sigmoid"]), "bias": rng.choice([0.0, 0.02, 0.2]),
                "groups": groups, "top_groups": top, "pair": rng.random() < 0.5, "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.0, 0.1, 0.9])}
    if op == "rms":
        T, H = _log_int(rng, 2, 16383), _log_int(rng, 64, 7160)
        if rng.random() < 0.7:
            H = H // 8 * 8
        c = {"op": op, "dir": rng.choice(["forward", "forward", "backward"]), "T": T | 1 if T > 512 else T, "H": H,
             "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.7}
        if c["dir"] == "forward":
            c["out"] = rng.choice(["same", "row", "block", "mx"])
        elif c["T"] > 8192:
            c["T"] = c["T"] // 2 | 1
        return c
    while True:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c = {"op": op, "H": _log_int(rng, 64, 4096), "I": _log_int(rng, 64, 2048), "E": _log_int(rng, 1, 128),
             "dtype": dtype, "master": dtype == "bf16" and rng.random() < 0.5, "bits": rng.choice([32, 8])}
        if rng.random() < 0.7:
            c["H"], c["I"] = c["H"] // 8 * 8, c["I"] // 8 * 8
        if sum(_sizes(c)) <= 64 * 4700000:
            return c


# ---- inputs -----------------------------------------------------------------------------------------------------

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _sizes(case):
    """The parameters of one layer: the norm's weight, the gate, and each expert's two matrices."""
    h, i, e = case["H"], case["I"], case["E"]
    return [h, e * h] + [2 * i * h, h * i] * e


def _starts(sizes):
    """Where each tensor starts in one buffer: on blocks of the states, zeros between."""
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // STATE_BLOCK) * STATE_BLOCK
    return starts, at


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        T, E, K, dt = case["T"], case["E"], case["K"], DTYPES[case["dtype"]]
        # a spread for each token, and experts that are more popular than others
        logits = torch.randn(T, E, generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
        if case["masked"]:
            off = torch.rand(E, generator=gen, device="cuda") < case["masked"]
            logits = logits.masked_fill(off, -math.inf)
        s["logits"] = logits.to(dt)
        s["b"] = case["bias"] * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
        if case["dir"] == "backward":
            top, ids = s["logits"].float().topk(K, dim=1)
            s["ids"] = torch.where(torch.isfinite(top), ids, -1).to(torch.int32).contiguous()
            s["dw"] = torch.randn(T, K, generator=gen, device="cuda")
        if own:
            from nvfp4_mixture_experts_router_gb300 import api
            s["rule"] = api.RouteRule(score=api.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else api.MOE_SCORE_SOFTMAX,
                                      groups=case["groups"], topk_groups=case["top_groups"],
                                      group_score=api.MOE_GROUP_TOP2 if case["pair"] else api.MOE_GROUP_MAX,
                                      renormalize=case["renorm"], scale=case["scale"])
            if case["dir"] == "forward":
                s["ids"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
                s["w"] = torch.empty(T, K, dtype=torch.float32, device="cuda")
            else:
                s["dlogits"] = torch.empty(T, E, dtype=dt, device="cuda")
    elif case["op"] == "rms":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        # a residual stream: a spread for each channel, and a branch's output of the same type to add
        spread = 0.5 + torch.rand(H, generator=gen, device="cuda")
        s["x"] = (torch.randn(T, H, generator=gen, device="cuda") * spread).to(dt)
        s["gamma"] = 1.0 + _normal(gen, (H,), torch.float32, 0.2)
        s["res"] = _normal(gen, (T, H), dt, 2.0) if case["residual"] else None
        if case["dir"] == "backward":
            s["dh"] = s["res"]
            s["dy"] = _normal(gen, (T, H), dt)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + RMS_EPS)
        if own:
            from nvfp4_mixture_experts_router_gb300 import api
            f32 = {"dtype": torch.float32, "device": "cuda"}
            s["h_out"] = torch.empty(T, H, dtype=dt, device="cuda")
            if case["dir"] == "backward":
                s["dgamma"] = torch.empty(H, **f32)
                s["ws"] = torch.empty(api.moe_nvfp4_rms_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
            elif case["out"] == "same":
                s["y_out"], s["rstd_out"] = torch.empty(T, H, dtype=dt, device="cuda"), torch.empty(T, **f32)
            else:
                s["q_out"] = torch.empty(T, H, dtype=F8, device="cuda")
                s["scales"] = (torch.empty(T, **f32) if case["out"] == "row" else
                               torch.empty(T, -(-H // 128), **f32) if case["out"] == "block" else
                               torch.empty(T, -(-H // 32), dtype=torch.float8_e8m0fnu, device="cuda"))
    else:
        dt, sizes = DTYPES[case["dtype"]], _sizes(case)
        starts, total = _starts(sizes)
        used = torch.zeros(total, dtype=torch.bool, device="cuda")
        for a, n in zip(starts, sizes):
            used[a:a + n] = True
        make = lambda scale: torch.randn(total, generator=gen, device="cuda") * scale * used      # noqa: E731
        p, size = make(0.02), 10.0 ** float(torch.rand((), generator=gen, device="cuda") - 5.0)
        s["g"] = make(size).to(dt)
        s["p"], s["w"] = p.to(dt), p.clone() if case["master"] else None
        # states some hundred steps on: the moving averages of gradients of that size
        m = make(0.3 * size)
        v = make(size).square() * 0.05 + 0.5 * size * size * used
        s["norm"] = (s["g"].float().square().sum().sqrt()).reshape(1)
        s["step"] = 300
        if case["bits"] == 32:
            s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
        else:
            s["m"], s["ms"] = _to_blocks(m, False)
            s["v"], s["vs"] = _to_blocks(v.sqrt(), True)
        if own:
            from nvfp4_mixture_experts_router_gb300 import api
            cut = lambda t: None if t is None else [t[a:a + n] for a, n in zip(starts, sizes)]      # noqa: E731
            scales = lambda t: None if t is None else [       # noqa: E731
                t[a // STATE_BLOCK:a // STATE_BLOCK + -(-n // STATE_BLOCK)] for a, n in zip(starts, sizes)]
            s["list"] = api.AdamWList(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]), scales(s["ms"]),
                                      scales(s["vs"]), cut(s["w"]))
            s["rule"] = api.AdamWRule(lr=ADAMW["lr"], beta1=ADAMW["beta1"], beta2=ADAMW["beta2"], eps=ADAMW["eps"],
                                      weight_decay=ADAMW["weight_decay"], max_norm=ADAMW["max_norm"], clip_eps=CLIP_EPS)
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    plain = {"route": _route_plain, "rms": _rms_plain, "adamw": _adamw_plain}
    kernels = {"route": _route_own, "rms": _rms_own, "adamw": _adamw_own}
    return (kernels if own else plain)[state["op"]](state)


def _route_own(s):
    from nvfp4_mixture_experts_router_gb300 import api
    if s["dir"] == "forward":
        api.moe_nvfp4_route_topk(s["logits"], s["b"], s["rule"], s["ids"], s["w"])
        return {"ids": s["ids"], "w": s["w"]}
    api.moe_nvfp4_route_topk_backward(s["logits"], s["ids"], s["dw"], s["rule"], s["dlogits"])
    return {"dlogits": s["dlogits"]}


def _route_plain(s):
    K = s["K"]
    if s["dir"] == "forward":
        l = s["logits"].double()
        l = torch.where(l > -math.inf, l, -math.inf).clamp(max=LARGEST)        # NaN and -inf: not to be chosen
        can = l > -math.inf
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300) if s["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
        with_bias = score
        choice = l
        if s["b"] is not None:
            b = s["b"].double()
            can = can & (b > -math.inf)
            choice = with_bias = score + b
        choice = torch.where(can, choice, -math.inf)
        if s["groups"] > 1:
            G = s["groups"]
            by_group = torch.where(can, with_bias if s["pair"] else choice, -math.inf).view(len(l), G, -1)
            best = by_group.sort(dim=2, descending=True).values[:, :, :2 if s["pair"] else 1]
            group = best[:, :, 0]
            if s["pair"] and best.shape[2] == 2:
                group = group + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0.0)
            order = group.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
            taken = torch.zeros_like(group, dtype=torch.bool).scatter_(1, order, True)
            choice = torch.where(taken[:, :, None], choice.view(len(l), G, -1), -math.inf).view_as(l)
        ranked = choice.sort(dim=1, descending=True, stable=True)
        ids, there = ranked.indices[:, :K], ranked.values[:, :K] > -math.inf
        if s["renorm"]:
            picked = torch.where(there, l.gather(1, ids), -math.inf)
            most = picked.amax(1, keepdim=True)
            most = torch.where(most > -math.inf, most, 0.0)
            if s["score"] == "softmax":
                part = torch.exp(picked - most)
            else:       # the scores times exp(-min(most, 0)): none of them all underflows
                part = torch.exp(picked.clamp(max=0.0) - most.clamp(max=0.0)) / (1.0 + torch.exp(-picked.abs()))
            w = part / part.sum(1, keepdim=True).clamp(min=1e-300)
        else:
            w = score.gather(1, ids)
        return {"ids": torch.where(there, ids, -1).int(), "w": torch.where(there, w * s["scale"], 0.0).float()}
    l, ids = s["logits"].float().clamp(max=LARGEST), s["ids"].long()
    there = ids >= 0
    at = ids.clamp(min=0)
    u = torch.where(there, s["dw"] * s["scale"], 0.0)
    picked = torch.where(there, l.gather(1, at), -math.inf)
    if s["score"] == "softmax" and not s["renorm"]:
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
        mean = (p.gather(1, at) * u).sum(1, keepdim=True)
        du = torch.zeros_like(l).scatter_add_(1, at, u)
        return {"dlogits": (p * (du - mean)).to(s["logits"].dtype)}
    most = picked.amax(1, keepdim=True)
    most = torch.where(most > -math.inf, most, 0.0)
    if s["score"] == "softmax":
        w = torch.exp(picked - most)
        slope = torch.ones_like(w)
    else:
        w = torch.exp(picked.clamp(max=0.0) - most.clamp(max=0.0)) / (1.0 + torch.exp(-picked.abs()))
        slope = 1.0 / (1.0 + torch.exp(picked))                              # 1 - sigmoid
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
        d = w * slope * (u - (w * u).sum(1, keepdim=True))
    else:
        d = u * slope / (1.0 + torch.exp(-picked))
    d = torch.where(there, d, 0.0)
    return {"dlogits": torch.zeros_like(l).scatter_add_(1, at, d).to(s["logits"].dtype)}


def _rms_own(s):
    from nvfp4_mixture_experts_router_gb300 import api
    if s["dir"] == "backward":
        api.moe_nvfp4_rms_norm_backward(s["dy"], s["dh"], s["x"], s["gamma"], s["rstd"], s["h_out"], s["dgamma"], s["ws"])
        return {"dx": s["h_out"], "dgamma": s["dgamma"]}
    h = s["h_out"] if s["residual"] else None
    if s["out"] == "same":
        api.moe_nvfp4_rms_norm(s["x"], s["res"], s["gamma"], RMS_EPS, h, s["y_out"], None, None, s["rstd_out"])
        r = {"y": s["y_out"], "rstd": s["rstd_out"]}
    else:
        api.moe_nvfp4_rms_norm(s["x"], s["res"], s["gamma"], RMS_EPS, h, None, s["q_out"], s["scales"])
        r = {"q": s["q_out"], "scales": s["scales"]}
    return {**r, "h": h} if s["residual"] else r


def _rms_plain(s):
    dt = s["x"].dtype
    T, H = s["x"].shape
    x = s["x"].float()
    if s["dir"] == "backward":
        dy = s["dy"].float()
        hat = x * s["rstd"][:, None]
        g = dy * s["gamma"]
        dx = s["rstd"][:, None] * (g - hat * (g * hat).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dgamma": (dy * hat).sum(0)}
    r = {}
    if s["residual"]:
        r["h"] = (x + s["res"].float()).to(dt)
        x = r["h"].float()
    rstd = torch.rsqrt((x * x).mean(1) + RMS_EPS)
    y = x * rstd[:, None] * s["gamma"]
    if s["out"] == "same":
        return {"y": y.to(dt), "rstd": rstd, **r}
    if s["out"] == "row":
        most = y.abs().amax(1)
        scale = torch.where(most > 0, most / F8_MAX, 1.0)
        return {"q": (y / scale[:, None]).clamp(-F8_MAX, F8_MAX).to(F8), "scales": scale, **r}
    n = 128 if s["out"] == "block" else 32
    blocks = torch.nn.functional.pad(y, (0, -H % n)).view(T, -1, n)
    most = blocks.abs().amax(2)
    if s["out"] == "block":
        scale = torch.where(most > 0, most / F8_MAX, 1.0)
    else:       # the power of two that takes the largest magnitude into [256, 512)
        power = torch.where(most > 0, torch.frexp(most).exponent - 9, -127).clamp(-127, 127)
        scale = torch.ldexp(torch.ones_like(most), power)
    q = (blocks / scale[:, :, None]).clamp(-F8_MAX, F8_MAX).to(F8)
    return {"q": q.view(T, -1)[:, :H].contiguous(), "scales": scale.to(torch.float8_e8m0fnu) if n == 32 else scale, **r}


def _to_blocks(t, positive):
    """Values in E4M3 with a scale for each block; of roots of second moments (`positive`) none but zero becomes zero."""
    blocks = t.view(-1, STATE_BLOCK)
    most = blocks.abs().amax(1)
    keep = most >= STATE_FLUSH
    scale = torch.where(keep, most / F8_MAX, 0.0)
    q = torch.where(keep[:, None], blocks / torch.where(keep, scale, 1.0)[:, None], 0.0).clamp(-F8_MAX, F8_MAX)
    if positive:
        q = torch.where(q > 0, q.clamp(min=2.0 ** -9), q)
    return q.to(F8).view(-1), scale


def _of_blocks(q, scale):
    return (q.view(-1, STATE_BLOCK).float() * scale[:, None]).view(-1)


def _adamw_own(s):
    from nvfp4_mixture_experts_router_gb300 import api
    s["step"] += 1
    api.moe_nvfp4_adamw(s["list"], s["rule"], s["step"], s["norm"])
    return {k: s[k] for k in ("p", "w", "m", "v", "ms", "vs") if s[k] is not None}


def _adamw_plain(s):
    a = ADAMW
    s["step"] += 1
    clip = (a["max_norm"] / (s["norm"] + CLIP_EPS)).clamp(max=1.0)
    g = s["g"].float() * clip
    m, v = s["m"], s["v"]
    if s["bits"] == 8:
        m, v = _of_blocks(m, s["ms"]), _of_blocks(v, s["vs"]).square()
    m.mul_(a["beta1"]).add_(g, alpha=1.0 - a["beta1"])
    v.mul_(a["beta2"]).add_(g * g, alpha=1.0 - a["beta2"])
    rate = a["lr"] / (1.0 - a["beta1"] ** s["step"])
    over = (v / (1.0 - a["beta2"] ** s["step"])).sqrt().add_(a["eps"])
    p = s["w"] if s["w"] is not None else s["p"].float()
    p = p * (1.0 - a["lr"] * a["weight_decay"]) - rate * (m / over)
    if s["w"] is not None:
        s["w"].copy_(p)
    s["p"].copy_(p)
    if s["bits"] == 8:
        for name, t, positive in (("m", m, False), ("v", v.sqrt(), True)):
            q, scale = _to_blocks(t, positive)
            s[name].copy_(q)
            s[name + "s"].copy_(scale)
    return {k: s[k] for k in ("p", "w", "m", "v", "ms", "vs") if s[k] is not None}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "route":
        T, E, K = case["T"], case["E"], case["K"]
        if case["dir"] == "forward":
            return {"bytes": T * E * b + 8 * T * K + (4 * E if case["bias"] else 0), "flops": 5.0 * T * E}
        full = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * b + 8 * T * K + T * (E if full else K) * b, "flops": (5.0 if full else 1.0) * T * E}
    if case["op"] == "rms":
        n, rows = case["T"] * case["H"], 1 + (case["residual"] is True)
        if case["dir"] == "backward":
            return {"bytes": n * b * (rows + 2) + 8 * case["H"] + 4 * case["T"], "flops": 9.0 * n}
        out = {"same": b * n + 4 * case["T"], "row": n + 4 * case["T"], "block": n + n // 32, "mx": n + n // 32}
        kept = b * n * (2 * rows - 1)       # x; and the residual and the sum
        return {"bytes": kept + out[case["out"]] + 4 * case["H"], "flops": 5.0 * n}
    n = sum(_sizes(case))
    each = b + (2 * b if not case["master"] else b + 8) + (16 if case["bits"] == 32 else 4 + 16 / STATE_BLOCK)
    return {"bytes": n * each, "flops": 15.0 * n}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def _e4m3(x):
    """x rounded to E4M3, half to even, in 64 bits."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(x), e - 4)
    return (torch.round(x / step) * step).clamp(-F8_MAX, F8_MAX)


def _chosen(s, l):
    """The experts of each token, one after the other (-1: none left)."""
    E, G = s["E"], s["groups"]
    p = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l.clamp(min=-1e30), 1)
    c = l if s["b"] is None else p + s["b"].double()
    c = c.masked_fill(l == -math.inf, -math.inf)
    if G > 1:
        of_group = p.masked_fill(l == -math.inf, -math.inf) if s["pair"] and s["b"] is None else c
        first, second = of_group.view(-1, G, E // G), None
        best = first.max(2)
        value = best.values
        if s["pair"]:
            second = first.scatter(2, best.indices[:, :, None], -math.inf).amax(2)
            value = value + torch.where(second == -math.inf, 0.0, second)
        out = torch.ones_like(value, dtype=torch.bool)
        for _ in range(s["top_groups"]):
            g = value.argmax(1, keepdim=True)
            out.scatter_(1, g, False)
            value = value.scatter(1, g, -math.inf)
        c = c.masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
    ids = []
    for _ in range(s["K"]):
        i = c.argmax(1, keepdim=True)
        ids.append(torch.where(c.gather(1, i) == -math.inf, -1, i))
        c = c.scatter(1, i, -math.inf)
    return torch.cat(ids, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        l = s["logits"].double()
        if s["dir"] == "forward":
            ids = _chosen(s, l)
            there, at = ids >= 0, ids.clamp(min=0)
            if s["score"] == "softmax":
                log_score = torch.log_softmax(l, 1) if not s["masked"] else torch.log_softmax(l.clamp(min=-1e30), 1)
            else:
                log_score = torch.nn.functional.logsigmoid(l)
            picked = torch.where(there, log_score.gather(1, at), -math.inf)
            if s["renorm"]:
                picked = picked - torch.logsumexp(picked, 1, keepdim=True)
            return {"ids": None, "w": torch.where(there, torch.exp(picked) * s["scale"], 0.0)}
        # the gradient of sum(dw * w) by differentiation
        l = l.clamp(min=-1e30).requires_grad_(True)
        there, at = s["ids"] >= 0, s["ids"].long().clamp(min=0)
        log_score = torch.log_softmax(l, 1) if s["score"] == "softmax" else torch.nn.functional.logsigmoid(l)
        picked = torch.where(there, log_score.gather(1, at), -1e30)
        if s["renorm"]:
            picked = picked - torch.logsumexp(picked, 1, keepdim=True)
        w = torch.where(there, torch.exp(picked) * s["scale"], 0.0)
        return {"dlogits": torch.autograd.grad((w * s["dw"].double()).sum(), l)[0]}
    if case["op"] == "rms":
        x = s["x"].double()
        T, H = x.shape
        if case["dir"] == "backward":
            x.requires_grad_(True)
            gamma = s["gamma"].double().requires_grad_(True)
            y = x / (x.square().sum(1, keepdim=True) / H + RMS_EPS).sqrt() * gamma
            dx, dgamma = torch.autograd.grad((y * s["dy"].double()).sum(), [x, gamma])
            return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dgamma": dgamma}
        r = {}
        if s["residual"]:
            x = x + s["res"].double()
            r["h"] = x
            x = x.to(s["x"].dtype).double()           # the norm is that of the sum as it is kept
        rstd = 1.0 / (torch.linalg.vector_norm(x, dim=1) ** 2 / H + RMS_EPS).sqrt()
        y = x * (rstd[:, None] * s["gamma"].double())
        if case["out"] == "same":
            return {"y": y, "rstd": rstd, **r}
        n = {"row": H, "block": 128, "mx": 32}[case["out"]]
        group = torch.arange(H, device="cuda") // n
        most = torch.zeros(T, -(-H // n), dtype=torch.float64, device="cuda")
        most.scatter_reduce_(1, group.expand(T, H), y.abs(), "amax")
        scale = most / F8_MAX if case["out"] != "mx" else 2.0 ** (torch.floor(torch.log2(most)) - 8)
        q = _e4m3(y / scale[:, group])
        return {"q": q, "scales": scale.view(T) if case["out"] == "row" else scale, **r}
    a, step = ADAMW, s["step"] + 1
    block = torch.arange(len(s["p"]), device="cuda") // STATE_BLOCK
    g = s["g"].double() * min(1.0, a["max_norm"] / (float(s["norm"]) + CLIP_EPS))
    m, v = s["m"].to(torch.float64), s["v"].to(torch.float64)
    if case["bits"] == 8:
        m, v = m * s["ms"].double()[block], (v * s["vs"].double()[block]) ** 2
    m = torch.lerp(g, m, a["beta1"])
    v = torch.lerp(g * g, v, a["beta2"])
    del g
    p = (s["w"] if s["w"] is not None else s["p"]).double()
    p = p - a["lr"] * (a["weight_decay"] * p + m / (1 - a["beta1"] ** step) /
                       ((v / (1 - a["beta2"] ** step)).sqrt() + a["eps"]))
    r = {"p": p, "m": m, "v": v}
    if case["master"]:
        r["w"] = p
    if case["bits"] == 8:
        v.sqrt_()
        for name in ("m", "v"):
            most = r[name].abs().view(-1, STATE_BLOCK).amax(1)
            r[name + "s"] = most / F8_MAX
            q = _e4m3(r[name] / r[name + "s"].clamp(min=1e-300)[block])
            r[name] = torch.where((r[name] > 0) & (q == 0), 2.0 ** -9, q) if name == "v" else q
    return r
