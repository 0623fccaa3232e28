"""The operators around the VQ products of a feed-forward block, as they are measured: expert routing, e4m3
quantization and the block-scaled e4m3 product, and the fused norms.

`run` computes a case in plain torch operations (`own = False`) or through this package's entry points
(`own = True`); `exact` computes it once more from its definition in 64 bits.
"""

import math

import torch

own = False

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
DTYPES = {"fp16": F16, "bf16": BF16, "fp32": F32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128          # columns (and weight rows) that share a scale
E4M3_MAX = 448.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _route(name, T, E, k, score, dtype, bias=False, groups=1, top_groups=1, group_score="max", renorm=True,
           scale=1.0, masked=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "dtype": dtype, "bias": bias,
            "groups": groups, "top_groups": top_groups, "group_score": group_score, "renorm": renorm,
            "scale": scale, "masked": masked}


def _quant(name, T, cols, dtype):
    return {"name": name, "op": "quant", "T": T, "cols": cols, "dtype": dtype}


def _product(name, T, rows, cols, y, epilogue="none"):
    return {"name": name, "op": "product", "T": T, "rows": rows, "cols": cols, "y": y, "epilogue": epilogue}


def _norm(name, T, cols, block, residual, out, post=True, gate="none", gate_act="none", alpha=1.0, beta=1.0,
          offset=0.0):
    return {"name": name, "op": "norm", "T": T, "cols": cols, "block": block, "residual": residual, "out": out,
            "post": post, "gate": gate, "gate_act": gate_act, "alpha": alpha, "beta": beta, "offset": offset}


def listed():
    return [
        # one decode token over the 256-expert, top-8 router of the routed workloads
        _route("route one token", 1, 256, 8, "softmax", "bf16"),
        # a long prefill chunk through a sigmoid router with a balance bias and expert groups
        _route("route prefill grouped", 16384, 256, 8, "sigmoid", "fp32", bias=True, groups=8, top_groups=4,
               group_score="top2", scale=2.5),
        # an odd chunk, an expert count off the wave width, padded tokens and switched-off experts
        _route("route odd masked", 1021, 160, 6, "softmax", "bf16", groups=8, top_groups=3, renorm=False,
               masked=True),
        # activations of a small decode batch entering the dense down projection
        _quant("quantize decode batch", 4, 17408, "bf16"),
        # a prefill chunk at the dense hidden size
        _quant("quantize prefill", 4096, 5120, "fp16"),
        # one decode token through a dense gate-sized projection kept in 8 bits
        _product("product one token", 1, 17408, 5120, "bf16"),
        # a small serving batch through the down projection
        _product("product 16 tokens", 16, 5120, 17408, "fp32"),
        # an odd chunk, odd rows and a partial last scale block
        _product("product odd", 197, 1001, 2000, "fp32"),
        # a prefill chunk through interleaved gate and up rows with the fused SwiGLU
        _product("product prefill swiglu", 2048, 17408, 5120, "bf16", epilogue="swiglu"),
        # one decode token between two layers: combine output in, next block's input out
        _norm("norm one token", 1, 5120, "fp32", "bf16", "bf16"),
        # a small odd chunk with a gate a channel, leaving e4m3 for the 8-bit product
        _norm("norm odd to e4m3", 333, 2000, "fp16", "fp32", "e4m3", gate="channel", gate_act="tanh", alpha=0.5,
              offset=1.0),
        # a prefill chunk with a sigmoid gate a token (a shared expert's) and a residual scale
        _norm("norm prefill", 4096, 5120, "bf16", "bf16", "bf16", gate="token", gate_act="sigmoid", alpha=0.25,
              beta=0.5),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quant", "product", "product", "norm"])
    if op == "route":
        T = _spread(rng, 1, 16384)
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        size = _spread(rng, max(2, 8 // groups), 256 // groups)
        E = groups * size
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * size))
        c = _route("", T, E, k, rng.choice(["softmax", "sigmoid"]), rng.choice(["fp32", "fp16", "bf16"]),
                   bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                   group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                   scale=rng.choice([1.0, 2.5, 0.5]), masked=rng.random() < 0.4)
    elif op == "quant":
        T = _spread(rng, 1, 4096)
        c = _quant("", T, 16 * _spread(rng, 1, min(1088, 4096 * 5120 // T // 16)), rng.choice(["fp16", "bf16"]))
    elif op == "product":
        T = _spread(rng, 1, 2048)
        epi = "swiglu" if rng.random() < 0.3 else "none"
        rows = _spread(rng, 16, 17408)
        rows += rows % 2 if epi == "swiglu" else 0
        cols = 16 * _spread(rng, 2, min(1088, 17408 * 5120 // rows // 16))
        c = _product("", T, rows, cols, rng.choice(["fp32", "fp16", "bf16"]), epi)
    else:
        T = _spread(rng, 1, 4096)
        out = rng.choice(["fp16", "bf16", "e4m3"])
        unit = 16 if out == "e4m3" else 1
        cols = unit * _spread(rng, max(1, 64 // unit), min(17408, 4096 * 5120 // T) // unit)
        f = rng.choice(["fp16", "bf16"])
        c = _norm("", T, cols, rng.choice(["fp32", f]), rng.choice(["fp32", f]), f if out != "e4m3" else out,
                  post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token", "full"]),
                  gate_act=rng.choice(["none", "sigmoid", "tanh"]), alpha=rng.choice([1.0, 0.5, 0.22]),
                  beta=rng.choice([1.0, 0.7]), offset=rng.choice([0.0, 1.0]))
    del c["name"]
    return c


def work(case):
    c = case
    size = {"fp16": 2, "bf16": 2, "fp32": 4, "e4m3": 1}
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * size[c["dtype"]] + c["T"] * c["k"] * 8 + (4 * c["E"] if c["bias"] else 0),
                "flops": 10 * n}
    if c["op"] == "quant":
        n, blocks = c["T"] * c["cols"], c["T"] * -(-c["cols"] // BLOCK)
        return {"bytes": 3 * n + 4 * blocks, "flops": 2 * n}
    if c["op"] == "product":
        T, R, C = c["T"], c["rows"], c["cols"]
        kb = -(-C // BLOCK)
        out = T * (R // 2 if c["epilogue"] == "swiglu" else R) * size[c["y"]]
        return {"bytes": T * C + R * C + 4 * kb * (T + -(-R // BLOCK)) + out, "flops": 2 * T * R * C}
    n = c["T"] * c["cols"]
    gate = {"none": 0, "channel": c["cols"], "token": c["T"], "full": n}[c["gate"]]
    b = n * (size[c["block"]] + 2 * size[c["residual"]] + size[c["out"]]) + 2 * gate
    b += 2 * c["cols"] * (2 if c["post"] else 1)
    if c["out"] == "e4m3":
        b += 4 * c["T"] * -(-c["cols"] // BLOCK)
    return {"bytes": b, "flops": 12 * n}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _activations(g, T, cols):
    """fp32 N(0, 1) with one channel in 64 twenty times larger, as hidden states have."""
    x = torch.randn(T, cols, device="cuda", generator=g)
    hot = torch.rand(cols, device="cuda", generator=g) < 1 / 64
    return torch.where(hot, 20 * x, x)


def _split(x, rows, cols):
    """x [R][C] padded with zeros to whole blocks of rows x cols, as [R/rows][rows][C/cols][cols]."""
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, -C % cols, 0, -R % rows))
    return x.reshape(x.shape[0] // rows, rows, x.shape[1] // cols, cols)


def _stored(x, rows):
    """Values and scales of an e4m3 tensor as a checkpoint or an earlier step leaves them (blocks of rows x 128)."""
    R, C = x.shape
    b = _split(x, rows, BLOCK)
    s = b.abs().amax((1, 3), keepdim=True).clamp_min(1e-30) / E4M3_MAX
    q = (b / s).clamp(-E4M3_MAX, E4M3_MAX).reshape(b.shape[0] * rows, -1)[:R, :C]
    return q.contiguous().to(E4M3), s[:, 0, :, 0].contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        # a few experts are popular: logits of spread 1.5 around per-expert means
        x = 1.5 * torch.randn(T, E, device="cuda", generator=g) + torch.randn(E, device="cuda", generator=g)
        x = x.to(DTYPES[c["dtype"]])
        if c["masked"]:
            off = torch.rand(E, device="cuda", generator=g) < 0.1      # experts off for this batch
            x[:, off] = torch.finfo(x.dtype).min
            x[torch.rand(T, E, device="cuda", generator=g) < 0.05] = -math.inf
            x[torch.rand(T, device="cuda", generator=g) < 0.05] = -math.inf   # padded tokens
        s["logits"] = x
        s["bias"] = 0.05 * torch.randn(E, device="cuda", generator=g) if c["bias"] else None
    elif c["op"] == "quant":
        s["x"] = _activations(g, c["T"], c["cols"]).to(DTYPES[c["dtype"]])
    elif c["op"] == "product":
        s["x"], s["x_scales"] = _stored(_activations(g, c["T"], c["cols"]), 1)
        s["w"], s["w_scales"] = _stored(0.02 * torch.randn(c["rows"], c["cols"], device="cuda", generator=g), BLOCK)
    else:
        T, C = c["T"], c["cols"]
        dt = F16 if "fp16" in (c["block"], c["residual"], c["out"]) else BF16   # the model's 16-bit type
        s["block"] = (0.3 * _activations(g, T, C)).to(DTYPES[c["block"]])
        s["residual"] = _activations(g, T, C).to(DTYPES[c["residual"]])
        weight = lambda: ((1 - c["offset"]) + 0.1 * torch.randn(C, device="cuda", generator=g)).to(dt)  # noqa: E731
        s["pre"] = weight()
        s["post"] = weight() if c["post"] else None
        shape = {"none": None, "channel": (C,), "token": (T, 1), "full": (T, C)}[c["gate"]]
        s["gate"] = None if shape is None else torch.randn(shape, device="cuda", generator=g).to(dt)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _round_e4m3(v):
    """fp64 v rounded to e4m3 values, ties to even: 3 bits behind the leading one, steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _plain_quant(x):
    T, C = x.shape
    b = _split(x.float(), 1, BLOCK)
    amax = b.abs().amax((1, 3), keepdim=True)
    s = torch.where(amax > 0, (amax.double() / E4M3_MAX).float(), 1.0)   # rounded once, not by a reciprocal
    q = _round_e4m3(b.double() / s.double()).reshape(T, -1)[:, :C]   # in 64 bits: quotients lie next to ties
    return q.float().to(E4M3), s[:, 0, :, 0].contiguous()


def _plain_route(c, logits, bias):
    T, E = logits.shape
    x = logits.double()                       # in 64 bits: keys lie next to each other at the border of the choice
    dead = x.isnan() | (x == -math.inf)
    if bias is not None:
        dead = dead | bias.isnan() | (bias == -math.inf)
    x = x.clamp(-torch.finfo(F32).max, torch.finfo(F32).max)
    if c["score"] == "softmax":
        m = x.masked_fill(dead, -math.inf).amax(1, keepdim=True)
        p = torch.where(dead, 0.0, torch.exp(x - torch.where(m == -math.inf, 0.0, m)))
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    else:
        p = torch.where(dead, 0.0, 1 / (1 + torch.exp(-x)))
    key = (x if bias is None else p + bias.double()).masked_fill(dead, -math.inf)
    G = c["groups"]
    if G > 1:
        if c["group_score"] == "max":
            score = key.reshape(T, G, -1).amax(2)
        else:
            v = (p if bias is None else key).masked_fill(dead, -math.inf).reshape(T, G, -1)
            v = v.sort(dim=2, descending=True).values
            score = v[:, :, 0] + torch.where(v[:, :, 1] == -math.inf, 0.0, v[:, :, 1])
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    best = key.sort(dim=1, descending=True, stable=True)
    ids, gone = best.indices[:, :c["k"]], best.values[:, :c["k"]] == -math.inf
    w = torch.where(gone, 0.0, p.gather(1, ids))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return {"ids": ids.masked_fill(gone, -1).int(), "weights": (w * c["scale"]).float()}


def _scaled(q, s, rows):
    """The fp32 values of an e4m3 tensor with a scale for each block of rows x 128."""
    R, C = q.shape
    b = _split(q.float(), rows, BLOCK) * s[:, None, :, None]
    return b.reshape(b.shape[0] * rows, -1)[:R, :C]


def _plain_product(c, s):
    y = _scaled(s["x"], s["x_scales"], 1) @ _scaled(s["w"], s["w_scales"], BLOCK).t()
    if c["epilogue"] == "swiglu":
        a, b = y[:, 0::2], y[:, 1::2]
        y = a / (1 + torch.exp(-a)) * b
    return {"y": y.to(DTYPES[c["y"]])}


def _plain_norm(c, s):
    u = s["block"].float()
    if c["post"]:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + 1e-6) * (s["post"].float() + c["offset"])
    if s["gate"] is not None:
        a = s["gate"].float()
        a = 1 / (1 + torch.exp(-a)) if c["gate_act"] == "sigmoid" else torch.tanh(a) if c["gate_act"] == "tanh" else a
        u = u * a
    v = c["beta"] * s["residual"].float() + c["alpha"] * u
    h = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * (s["pre"].float() + c["offset"])
    out = {"residual": v.to(s["residual"].dtype)}
    if c["out"] == "e4m3":
        out["h"], out["h_scales"] = _plain_quant(h)
    else:
        out["h"] = h.to(DTYPES[c["out"]])
    return out


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _own(c, s):
    import vq_dequant_matmul_gemv_amd as vq
    if c["op"] == "route":
        router = vq.Router(c["E"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                           top_groups=c["top_groups"], group_score=c["group_score"], renormalize=c["renorm"],
                           scale=c["scale"])
        ids, weights = vq.moe_route(router, s["logits"])
        return {"ids": ids, "weights": weights}
    if c["op"] == "quant":
        q, scales = vq.fp8_quant(s["x"])
        return {"q": q, "scales": scales}
    if c["op"] == "product":
        w = vq.FP8Tensor(s["w"], s["w_scales"])
        return {"y": vq.fp8_gemm(w, s["x"], s["x_scales"], y_dtype=DTYPES[c["y"]],
                                 epilogue=None if c["epilogue"] == "none" else c["epilogue"])}
    v, h, scales = vq.norm(s["block"], s["residual"], post_weight=s["post"], pre_weight=s["pre"], gate=s["gate"],
                           gate_act=c["gate_act"], alpha=c["alpha"], beta=c["beta"], weight_offset=c["offset"],
                           eps=1e-6, h_dtype=E4M3 if c["out"] == "e4m3" else DTYPES[c["out"]])
    return {"residual": v, "h": h, "h_scales": scales} if c["out"] == "e4m3" else {"residual": v, "h": h}


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "route":
        return _plain_route(c, state["logits"], state["bias"])
    if c["op"] == "quant":
        q, scales = _plain_quant(state["x"])
        return {"q": q, "scales": scales}
    return (_plain_product if c["op"] == "product" else _plain_norm)(c, state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_quant(x):
    """x: fp64 [T][C], from which the scales (rounded to fp32) and the nearest e4m3 values follow."""
    table = torch.tensor([(i & 7 | (8 if i >> 3 else 0)) * 2.0 ** (max(i >> 3, 1) - 10) for i in range(127)],
                         dtype=torch.float64, device=x.device)
    middles = (table[1:] + table[:-1]) / 2
    q, scales = torch.empty_like(x), []
    for c0 in range(0, x.shape[1], BLOCK):
        part = x[:, c0:c0 + BLOCK]
        top = part.abs().max(1).values
        s = torch.where(top == 0, torch.ones_like(top), (top / 448).float().double())
        a = (part.abs() / s[:, None]).contiguous()
        low = torch.bucketize(a, middles)                  # ties go down
        up = torch.bucketize(a, middles, right=True)       # ties go up
        i = torch.where((low != up) & (low % 2 == 1), up, low)
        q[:, c0:c0 + BLOCK] = torch.copysign(table[i], part)
        scales.append(s)
    return q, torch.stack(scales, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        q, scales = _exact_quant(s["x"].double())
        return {"q": q, "scales": scales}
    if c["op"] == "product":
        T, R = c["T"], c["rows"]
        y = torch.zeros(T, R, dtype=torch.float64, device="cuda")
        for k in range(s["x_scales"].shape[1]):
            cut = slice(BLOCK * k, BLOCK * (k + 1))
            part = s["x"][:, cut].double() @ s["w"][:, cut].double().t()
            row_scale = s["w_scales"][:, k].double().repeat_interleave(BLOCK)[:R]
            y += part * s["x_scales"][:, k].double()[:, None] * row_scale[None, :]
        if c["epilogue"] == "swiglu":
            y = y.view(T, R // 2, 2)
            y = y[..., 0] * torch.sigmoid(y[..., 0]) * y[..., 1]
        return {"y": y}
    if c["op"] == "norm":
        v = s["block"].double()
        if c["post"]:
            v = v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / c["cols"] + 1e-6) * (s["post"].double() + c["offset"])
        if s["gate"] is not None:
            g = s["gate"].double()
            v = v * {"none": lambda t: t, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[c["gate_act"]](g)
        v = v * c["alpha"] + s["residual"].double() * c["beta"]
        h = v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / c["cols"] + 1e-6) * (s["pre"].double() + c["offset"])
        if c["out"] != "e4m3":
            return {"residual": v, "h": h}
        q, scales = _exact_quant(h)
        return {"residual": v, "h": q, "h_scales": scales}
    # routing: one choice after the other, for all tokens at once
    x = s["logits"].double()
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    live = torch.isfinite(x) | (x == math.inf)
    if s["bias"] is not None:
        live &= (torch.isfinite(s["bias"]) | (s["bias"] == math.inf))[None]
    if c["score"] == "softmax":
        p = torch.softmax(torch.where(live, x, -math.inf), 1).nan_to_num(0.0)
    else:
        p = torch.sigmoid(x) * live
    rank_by = x if s["bias"] is None else p + s["bias"].double()
    gone = torch.tensor(-math.inf, dtype=torch.float64, device="cuda")
    rank_by = torch.where(live, rank_by, gone)
    if G > 1:
        v = rank_by if (s["bias"] is not None or c["group_score"] == "max") else torch.where(live, p, gone)
        v = v.view(T, G, E // G)
        first = v.max(2)
        score = first.values.clone()
        if c["group_score"] == "top2":
            rest = v.scatter(2, first.indices[..., None], -math.inf).max(2).values
            score += torch.where(rest > -math.inf, rest, torch.zeros_like(rest))
        allowed = torch.zeros(T, G, dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):                   # the best group left, the lowest of equals
            left = torch.where(allowed, gone, score)
            top = left.max(1, keepdim=True).values
            pick = ((left == top) & ~allowed).int().argmax(1)
            allowed[torch.arange(T, device="cuda"), pick] = True
        rank_by = torch.where(allowed.repeat_interleave(E // G, 1), rank_by, gone)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    at = torch.arange(T, device="cuda")
    rank_by = rank_by.clone()
    for j in range(k):
        top = rank_by.max(1).values
        pick = (rank_by == top[:, None]).int().argmax(1)
        some = top > -math.inf
        ids[:, j] = torch.where(some, pick, torch.full_like(pick, -1)).int()
        w[:, j] = torch.where(some, p[at, pick], torch.zeros_like(top))
        rank_by[at, pick] = -math.inf
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return {"ids": ids, "weights": w * c["scale"]}
