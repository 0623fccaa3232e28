"""Microscaled 4-bit tensors (e2m1 values, a power-of-two scale for each 32 columns) as they are measured: quantizing
activations and reading them back, the product, and a whole mixture-of-experts layer for a few tokens.

`run` computes a case in plain torch operations (`own = False`) or through this package's entry points
(`own = True`); `exact` computes it once more from its definition in 64 bits.
"""

import math

import torch

own = False

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
DTYPES = {"fp16": F16, "bf16": BF16, "fp32": F32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
BLOCK = 32           # columns that share a scale


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _quant(name, T, cols, dtype):
    return {"name": name, "op": "quant", "T": T, "cols": cols, "dtype": dtype}


def _product(name, T, rows, cols, x, y, epilogue="none"):
    return {"name": name, "op": "product", "T": T, "rows": rows, "cols": cols, "x": x, "y": y, "epilogue": epilogue}


def _moe(name, T, E, k, hidden, inter, dtype, y, score="softmax", bias=False, groups=1, top_groups=1, renorm=True,
         scale=1.0, masked=False):
    return {"name": name, "op": "moe", "T": T, "E": E, "k": k, "hidden": hidden, "inter": inter, "dtype": dtype,
            "y": y, "score": score, "bias": bias, "groups": groups, "top_groups": top_groups, "renorm": renorm,
            "scale": scale, "masked": masked}


def listed():
    return [
        # activations of a small decode batch entering the dense down projection
        _quant("quantize decode batch", 4, 17408, "bf16"),
        # a small odd chunk of fp32 values: weights of a small layer on their way into the format
        _quant("quantize odd fp32", 333, 2016, "fp32"),
        # a prefill chunk at the dense hidden size
        _quant("quantize prefill", 4096, 5120, "fp16"),
        # one decode token, its activations left in 16 bits, through a dense gate-sized projection
        _product("product one token", 1, 17408, 5120, "bf16", "bf16"),
        # a small serving batch through the down projection, both operands in 4 bits
        _product("product 16 tokens", 16, 5120, 17408, "mx4", "fp32"),
        # a larger odd decode batch with 16-bit activations, odd rows
        _product("product 61 tokens 16-bit x", 61, 5121, 4096, "fp16", "fp16"),
        # an odd chunk, odd rows, columns that end inside a group of blocks
        _product("product odd", 197, 1001, 2016, "mx4", "fp32"),
        # a prefill chunk through interleaved gate and up rows with the fused SwiGLU
        _product("product prefill swiglu", 2048, 17408, 5120, "mx4", "bf16", epilogue="swiglu"),
        # one decode token through the 256-expert, top-8 layer of the routed workloads
        _moe("moe one token", 1, 256, 8, 4096, 1024, "bf16", "bf16"),
        # five tokens, two of them padding, experts switched off, sizes off every tile, fp32 result
        _moe("moe odd masked", 5, 60, 4, 1504, 352, "fp16", "fp32", renorm=False, masked=True),
        # a small serving batch through a sigmoid router with a balance bias and expert groups
        _moe("moe 16 tokens grouped", 16, 256, 8, 4096, 1024, "bf16", "bf16", score="sigmoid", bias=True, groups=8,
             top_groups=4, scale=2.5),
        # a larger decode batch through the smaller routed workload
        _moe("moe 64 tokens", 64, 256, 8, 2048, 512, "bf16", "bf16"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "moe", "moe"])
    if op == "quant":
        T = _spread(rng, 1, 4096)
        cols = BLOCK * _spread(rng, 1, max(1, min(544, 4096 * 5120 // T // BLOCK)))
        c = _quant("", T, cols, rng.choice(["fp16", "bf16", "fp32"] if T <= 2048 else ["fp16", "bf16"]))
    elif op == "product":
        x = rng.choice(["mx4", "mx4", "fp16", "bf16"])
        T = _spread(rng, 1, 2048 if x == "mx4" else 128)
        epi = "swiglu" if rng.random() < 0.3 else "none"
        rows = _spread(rng, 16, 17408)
        rows += rows % 2 if epi == "swiglu" else 0
        cols = BLOCK * _spread(rng, 1, min(544, 17408 * 5120 // rows // BLOCK))
        c = _product("", T, rows, cols, x, rng.choice(["fp32", "fp16", "bf16"]), epi)
    else:
        T = _spread(rng, 1, 64)
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _spread(rng, max(1, 4 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, top_groups * size))
        hidden = BLOCK * _spread(rng, 2, 128)
        inter = BLOCK * _spread(rng, 1, max(1, min(32, 64 * 8 * 2048 * 512 // (T * k * hidden) // BLOCK)))
        c = _moe("", T, groups * size, k, hidden, inter, rng.choice(["fp16", "bf16"]),
                 rng.choice(["fp32", "fp16", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                 bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, renorm=rng.random() < 0.7,
                 scale=rng.choice([1.0, 2.5, 0.5]), masked=rng.random() < 0.4)
    del c["name"]
    return c


def _stored_bytes(rows, cols):
    return rows * cols // 2 + rows * cols // BLOCK


def work(case):
    c = case
    if c["op"] == "quant":    # read and quantized, then read back
        n = c["T"] * c["cols"]
        return {"bytes": 2 * n * SIZE[c["dtype"]] + 2 * _stored_bytes(c["T"], c["cols"]), "flops": 4 * n}
    if c["op"] == "product":
        T, R, C = c["T"], c["rows"], c["cols"]
        x = _stored_bytes(T, C) if c["x"] == "mx4" else 2 * T * C
        out = T * (R // 2 if c["epilogue"] == "swiglu" else R) * SIZE[c["y"]]
        return {"bytes": x + _stored_bytes(R, C) + out, "flops": 2 * T * R * C}
    T, E, k, H, I = c["T"], c["E"], c["k"], c["hidden"], c["inter"]
    hit = E * (1 - (1 - k / E) ** T)                       # distinct experts of evenly spread choices
    weights = hit * (_stored_bytes(2 * I, H) + _stored_bytes(H, I))
    other = T * E * SIZE[c["dtype"]] + T * H * (2 + SIZE[c["y"]]) + 8 * T * k + (4 * E if c["bias"] else 0)
    return {"bytes": weights + other, "flops": 6 * T * k * H * I}


# --------------------------------------------------------------------------
# the format in plain operations
# --------------------------------------------------------------------------

def _encode(x):
    """e2m1 codes [..][cols] and scale bytes [..][cols/32] of fp32 x [..][cols]: a block's scale is 2^(floor(log2 of
    its largest magnitude) - 2) (1 for a block of zeros), its values are the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6
    times the scale, ties to the even code, at most 6."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, 0).clamp(-127, 127)
    a = torch.ldexp(b.abs().double(), -e).clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    code = (torch.round(a / step) + torch.where(a < 2, 0, torch.where(a < 4, 2, 4))).to(torch.uint8)
    code = code | (torch.signbit(b).to(torch.uint8) << 3)
    return code.reshape(x.shape), (e.squeeze(-1) + 127).to(torch.uint8)


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _byte_values(device, dtype=F32):
    """The two values that each byte of codes stands for, [256][2]."""
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device, dtype=dtype)
    v = torch.cat([v, -v])
    byte = torch.arange(256, device=device)
    return torch.stack([v[byte % 16], v[byte // 16]], 1)


def _values(q, s):
    """fp32 values [..][cols] of packed codes [..][cols/2] and scale bytes [..][cols/32]."""
    v = _byte_values(q.device).index_select(0, q.reshape(-1).int())
    return (v.view(*s.shape, BLOCK) * torch.exp2(s.float() - 127).unsqueeze(-1)).view(*q.shape[:-1], -1)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _activations(g, T, cols):
    """fp32 N(0, 1) with one channel in 64 twenty times larger, as hidden states have."""
    x = torch.randn(T, cols, device="cuda", generator=g)
    hot = torch.rand(cols, device="cuda", generator=g) < 1 / 64
    return torch.where(hot, 20 * x, x)


def _stored(x):
    """Packed codes and scale bytes of a tensor as a checkpoint or an earlier step leaves them."""
    code, s = _encode(x)
    return _packed(code), s


def _stored_stack(g, E, rows, cols):
    """A stack of experts, a few at a time."""
    q = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, rows, cols // BLOCK, dtype=torch.uint8, device="cuda")
    some = max(1, (1 << 26) // (rows * cols))
    for e in range(0, E, some):
        w = 0.02 * torch.randn(min(some, E - e), rows, cols, device="cuda", generator=g)
        q[e:e + some], s[e:e + some] = _stored(w)
    return q, s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "quant":
        s["x"] = _activations(g, c["T"], c["cols"]).to(DTYPES[c["dtype"]])
    elif c["op"] == "product":
        x = _activations(g, c["T"], c["cols"])
        s["x"], s["x_scales"] = _stored(x) if c["x"] == "mx4" else (x.to(DTYPES[c["x"]]), None)
        s["w"], s["w_scales"] = _stored(0.02 * torch.randn(c["rows"], c["cols"], device="cuda", generator=g))
    else:
        T, E, H, I = c["T"], c["E"], c["hidden"], c["inter"]
        # a few experts are popular: logits of spread 1.5 around per-expert means
        x = 1.5 * torch.randn(T, E, device="cuda", generator=g) + torch.randn(E, device="cuda", generator=g)
        x = x.to(DTYPES[c["dtype"]])
        if c["masked"]:
            off = torch.rand(E, device="cuda", generator=g) < 0.1      # experts off for this batch
            x[:, off] = torch.finfo(x.dtype).min
            x[torch.rand(T, E, device="cuda", generator=g) < 0.05] = -math.inf
            x[torch.arange(T, device="cuda") % 5 >= 3] = -math.inf     # padded tokens
        s["logits"] = x
        s["bias"] = 0.05 * torch.randn(E, device="cuda", generator=g) if c["bias"] else None
        s["x"] = torch.randn(T, H, device="cuda", generator=g).to(DTYPES[c["dtype"]])   # a normed hidden state
        s["gate_up"], s["gate_up_scales"] = _stored_stack(g, E, 2 * I, H)
        s["down"], s["down_scales"] = _stored_stack(g, E, H, I)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _plain_quant(x):
    code, s = _encode(x.float())
    return {"values": _values(_packed(code), s).to(x.dtype), "scales": s.view(torch.float8_e8m0fnu)}


def _swiglu(y):
    a, b = y[..., 0::2], y[..., 1::2]
    return a / (1 + torch.exp(-a)) * b


def _plain_product(c, s):
    x = s["x"].float() if s["x_scales"] is None else _values(s["x"], s["x_scales"])
    y = x @ _values(s["w"], s["w_scales"]).t()
    return {"y": (_swiglu(y) if c["epilogue"] == "swiglu" else y).to(DTYPES[c["y"]])}


def _plain_route(c, logits, bias):
    T, E = logits.shape
    x = logits.double()                       # in 64 bits: keys lie next to each other at the border of the choice
    dead = x.isnan() | (x == -math.inf)
    if c["score"] == "softmax":
        m = x.masked_fill(dead, -math.inf).amax(1, keepdim=True)
        p = torch.where(dead, 0.0, torch.exp(x - torch.where(m == -math.inf, 0.0, m)))
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    else:
        p = torch.where(dead, 0.0, 1 / (1 + torch.exp(-x)))
    key = (x if bias is None else p + bias.double()).masked_fill(dead, -math.inf)
    G = c["groups"]
    if G > 1:                                 # groups by their two best
        v = (p if bias is None else key).masked_fill(dead, -math.inf).reshape(T, G, -1)
        v = v.sort(dim=2, descending=True).values
        score = v[:, :, 0]
        if v.shape[2] > 1:
            score = score + torch.where(v[:, :, 1] == -math.inf, 0.0, v[:, :, 1])
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    best = key.sort(dim=1, descending=True, stable=True)
    ids, gone = best.indices[:, :c["k"]], best.values[:, :c["k"]] == -math.inf
    w = torch.where(gone, 0.0, p.gather(1, ids))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return ids.masked_fill(gone, -1).int(), (w * c["scale"]).float()


def _plain_moe(c, s):
    T, k, H = c["T"], c["k"], c["hidden"]
    ids, weights = _plain_route(c, s["logits"], s["bias"])
    e = ids.clamp_min(0).reshape(-1).long()                # a choice of nothing has weight 0
    x = s["x"].float().repeat_interleave(k, 0).unsqueeze(2)
    h = _swiglu(torch.bmm(_values(s["gate_up"][e], s["gate_up_scales"][e]), x).squeeze(2))
    y = torch.bmm(_values(s["down"][e], s["down_scales"][e]), h.unsqueeze(2).contiguous())
    y = (y.view(T, k, H) * weights.unsqueeze(2)).sum(1)
    return {"y": y.to(DTYPES[c["y"]]), "ids": ids, "weights": weights}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _own(c, s):
    import vq_dequant_matmul_gemv_amd as vq
    if c["op"] == "quant":
        q, scales = vq.mx4_quant(s["x"])
        return {"values": vq.mx4_dequant(q, scales, dtype=s["x"].dtype), "scales": scales}
    if c["op"] == "product":
        return {"y": vq.mx4_gemm(vq.MX4Tensor(s["w"], s["w_scales"]), s["x"], s["x_scales"], y_dtype=DTYPES[c["y"]],
                                 epilogue=None if c["epilogue"] == "none" else c["epilogue"])}
    router = vq.Router(c["E"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                       top_groups=c["top_groups"], group_score="top2", renormalize=c["renorm"], scale=c["scale"])
    y, ids, weights = vq.mx4_moe(router, vq.MX4Tensor(s["gate_up"], s["gate_up_scales"]),
                                 vq.MX4Tensor(s["down"], s["down_scales"]), s["logits"], s["x"],
                                 y_dtype=DTYPES[c["y"]])
    return {"y": y, "ids": ids, "weights": weights}


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "quant":
        return _plain_quant(state["x"])
    return (_plain_product if c["op"] == "product" else _plain_moe)(c, state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_values(q, s):
    """fp64 values, digit by digit: sign, two bits of exponent, one of mantissa."""
    code = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1).to(torch.int16)
    e, m = (code >> 1) & 3, code & 1
    v = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * torch.exp2(e.double() - 1))
    v = torch.where(code >= 8, -v, v)
    return v * torch.exp2(s.double() - 127).repeat_interleave(BLOCK, -1)


def _exact_quant(x):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64, device=x.device)
    middles = (table[1:] + table[:-1]) / 2
    parts = x.double().split(BLOCK, dim=1)
    out, scales = [], []
    for p in parts:
        top = p.abs().max(1).values
        power = torch.floor(torch.log2(torch.where(top > 0, top, torch.full_like(top, 4.0))))
        power = torch.where(torch.exp2(power) > top, power - 1, power)      # a logarithm rounded up
        power = torch.where(torch.exp2(power + 1) <= top, power + 1, power)  # or down
        scale = torch.where(top > 0, torch.exp2(power - 2), torch.ones_like(top)).clamp_min(2.0 ** -127)
        a = (p.abs() / scale[:, None]).contiguous()
        low, up = torch.bucketize(a, middles), torch.bucketize(a, middles, right=True)
        i = torch.where((low != up) & (low % 2 == 1), up, low)
        out.append(torch.copysign(table[i], p) * scale[:, None])
        scales.append(scale)
    return {"values": torch.cat(out, 1), "scales": torch.stack(scales, 1)}


def _exact_route(c, s):
    """One choice after the other, for all tokens at once."""
    x = s["logits"].double()
    T, E, G = c["T"], c["E"], c["groups"]
    live = torch.isfinite(x)
    p = torch.sigmoid(x) * live if c["score"] == "sigmoid" else \
        torch.softmax(torch.where(live, x, -math.inf), 1).nan_to_num(0.0)
    gone = torch.tensor(-math.inf, dtype=F64, device="cuda")
    key = torch.where(live, x if s["bias"] is None else p + s["bias"].double(), gone)
    if G > 1:
        v = torch.where(live, p, gone) if s["bias"] is None else key
        v = v.view(T, G, E // G)
        first = v.max(2)
        rest = v.scatter(2, first.indices[..., None], -math.inf).max(2).values
        score = first.values + torch.where(rest > -math.inf, rest, torch.zeros_like(rest))
        allowed = torch.zeros(T, G, dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):                   # the best group left, the lowest of equals
            left = torch.where(allowed, gone, score)
            top = left.max(1, keepdim=True).values
            pick = ((left == top) & ~allowed).int().argmax(1)
            allowed[torch.arange(T, device="cuda"), pick] = True
        key = torch.where(allowed.repeat_interleave(E // G, 1), key, gone)
    ids = torch.full((T, c["k"]), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, c["k"], dtype=F64, device="cuda")
    at, key = torch.arange(T, device="cuda"), key.clone()
    for j in range(c["k"]):
        top = key.max(1).values
        pick = (key == top[:, None]).int().argmax(1)
        some = top > -math.inf
        ids[:, j] = torch.where(some, pick, torch.full_like(pick, -1)).int()
        w[:, j] = torch.where(some, p[at, pick], torch.zeros_like(top))
        key[at, pick] = -math.inf
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return ids, w * c["scale"]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        return _exact_quant(s["x"])
    if c["op"] == "product":
        x = s["x"].double() if c["x"] != "mx4" else _exact_values(s["x"], s["x_scales"])
        y = x @ _exact_values(s["w"], s["w_scales"]).t()
        if c["epilogue"] == "swiglu":
            y = y.view(c["T"], c["rows"] // 2, 2)
            y = y[..., 0] * torch.sigmoid(y[..., 0]) * y[..., 1]
        return {"y": y}
    ids, w = _exact_route(c, s)
    y = torch.zeros(c["T"], c["hidden"], dtype=F64, device="cuda")
    for e in sorted(set(ids[ids >= 0].tolist())):          # one expert after the other, with its tokens
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g = s["x"][t].double() @ _exact_values(s["gate_up"][e], s["gate_up_scales"][e]).t()
        h = g[:, 0::2] * torch.sigmoid(g[:, 0::2]) * g[:, 1::2]
        y.index_add_(0, t, w[t, j][:, None] * (h @ _exact_values(s["down"][e], s["down_scales"][e]).t()))
    return {"y": y, "ids": ids, "weights": w}
