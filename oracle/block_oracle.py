"""Plain CPU oracles (numpy, float64) of the operators around the VQ products.

TEST INFRASTRUCTURE ONLY, like vq_oracle: plain loops over the definitions in
include/vq.h, sharing no code with the GPU path.
"""

from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def route(logits, top_k, *, score="softmax", bias=None, groups=1, top_groups=1, group_score="max",
          renormalize=True, scale=1.0):
    """vq_moe_route of logits [T][E] (any float type): (ids int32 [T][k],
    weights float64 [T][k])."""
    x_all = np.asarray(logits, dtype=np.float64)
    T, E = x_all.shape
    ids = np.full((T, top_k), -1, dtype=np.int32)
    weights = np.zeros((T, top_k))
    b = None if bias is None else np.asarray(bias, dtype=np.float64)
    for t in range(T):
        x = x_all[t]
        live = ~np.isnan(x) & (x != -np.inf)
        if b is not None:
            live &= ~np.isnan(b) & (b != -np.inf)
        x = np.where(np.isnan(x), 0.0, np.clip(x, -F32_MAX, F32_MAX))
        p = np.zeros(E)
        if score == "softmax":
            if live.any():
                p[live] = np.exp(x[live] - x[live].max())
                p /= p.sum()
        else:
            with np.errstate(over="ignore"):
                p[live] = 1.0 / (1.0 + np.exp(-x[live]))
        key = x if b is None else p + b
        left = [e for e in range(E) if live[e]]
        if groups > 1:
            size = E // groups
            found = []
            for g in range(groups):
                mine = [e for e in left if e // size == g]
                if not mine:
                    continue
                if group_score == "max":
                    s = max(key[e] for e in mine)
                else:
                    s = sum(sorted((p[e] if b is None else key[e] for e in mine), reverse=True)[:2])
                found.append((-s, g))
            stay = {g for _, g in sorted(found)[:top_groups]}
            left = [e for e in left if e // size in stay]
        chosen = sorted(left, key=lambda e: (-key[e], e))[:top_k]
        w = np.array([p[e] for e in chosen])
        if renormalize and len(chosen):
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * scale
    return ids, weights


# ---------------------------------------------------------------------------
# e4m3 with a scale for each block of 128
# ---------------------------------------------------------------------------

BLOCK = 128

# value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits
E4M3 = np.array([(-1.0) ** (c >> 7) * (np.nan if (c & 0x7f) == 0x7f else
                                       (c & 7) * 2.0 ** -9 if ((c >> 3) & 15) == 0 else
                                       (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)])


def e4m3_nearest(v):
    """Codes (uint8) of the e4m3 values nearest to float64 v, ties to the even
    code, clamped to +-448; NaN and infinities give the NaN code 0x7f."""
    v = np.asarray(v, dtype=np.float64)
    bad = ~np.isfinite(v)
    a = np.minimum(np.abs(np.where(bad, 0.0, v)), 448.0)
    grid = E4M3[:127]
    up = np.clip(np.searchsorted(grid, a), 1, 126)       # grid[up - 1] < a <= grid[up] (but for a = 0)
    lo = up - 1
    dl, du = a - grid[lo], grid[up] - a                  # exact: both within a factor of 2, or small multiples
    code = np.where(dl < du, lo, np.where(du < dl, up, np.where(lo % 2 == 0, lo, up)))
    code = code | np.where(np.signbit(v), 0x80, 0)
    return np.where(bad, 0x7f, code).astype(np.uint8)


def fp8_quant(x):
    """(codes uint8 [T][C], scales fp32 [T][ceil(C/128)]) of x [T][C]."""
    x = np.asarray(x, dtype=np.float64)
    T, C = x.shape
    codes = np.zeros((T, C), dtype=np.uint8)
    scales = np.zeros((T, -(-C // BLOCK)), dtype=np.float32)
    for b in range(scales.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        amax = np.where(np.isfinite(part), np.abs(part), 0.0).max(axis=1)
        s = (amax / 448.0).astype(np.float32)
        s = np.where(s > 0, s, np.float32(1.0))
        scales[:, b] = s
        # the float64 quotient of an fp16/bf16 value and an fp32 scale lies on
        # a tie (5 bits) only if it is one: x = tie * s has at most 29 bits
        codes[:, b * BLOCK:(b + 1) * BLOCK] = e4m3_nearest(part / s.astype(np.float64)[:, None])
    return codes, scales


def fp8_values(codes, scales, rows=1):
    """float64 values of e4m3 codes [R][C] with a scale per rows x 128 block."""
    R, C = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), rows, axis=0)[:R], BLOCK, axis=1)[:, :C]
    return E4M3[codes] * s


def fp8_product(xc, xs, wc, ws):
    """(y [T][R], the sums of the magnitudes [T][R]) in float64."""
    x, w = fp8_values(xc, xs), fp8_values(wc, ws, BLOCK)
    return x @ w.T, np.abs(x) @ np.abs(w).T


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------

def norm(block=None, residual=None, *, post_weight=None, pre_weight=None, gate=None, gate_act=None, alpha=1.0,
         beta=1.0, weight_offset=0.0, eps=1e-6):
    """vq_norm in float64: dict of u (the scaled, gated block term), r (the
    residual term), v, rms (1 / rsqrt of v's mean square) and h."""
    f = lambda t: np.asarray(t, dtype=np.float64)  # noqa: E731
    u = r = 0.0
    if block is not None:
        u = f(block)
        if post_weight is not None:
            u = u / np.sqrt((u * u).mean(axis=1, keepdims=True) + eps) * (f(post_weight) + weight_offset)
        if gate is not None:
            g = f(gate)
            u = u * (1 / (1 + np.exp(-g)) if gate_act == "sigmoid" else np.tanh(g) if gate_act == "tanh" else g)
        u = alpha * u
    if residual is not None:
        r = beta * f(residual)
    v = u + r
    rms = np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    w = 1.0 if pre_weight is None else f(pre_weight) + weight_offset
    return {"u": u * np.ones_like(v), "r": r * np.ones_like(v), "v": v, "rms": rms, "w": w, "h": v / rms * w}


# ---------------------------------------------------------------------------
# e2m1 with a power-of-two scale for each 32 columns
# ---------------------------------------------------------------------------

MX4_BLOCK = 32
# value of every e2m1 code: sign, 2 exponent bits (bias 1), 1 mantissa bit
E2M1 = np.array([(-1.0) ** (c >> 3) * ((c & 1) * 0.5 if ((c >> 1) & 3) == 0 else
                                       (2 + (c & 1)) * 2.0 ** (((c >> 1) & 3) - 2)) for c in range(16)])


def e2m1_nearest(v):
    """Codes (uint8) of the e2m1 values nearest to finite float64 v, ties to
    the even code, clamped to +-6."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 6.0)
    grid = E2M1[:8]
    up = np.clip(np.searchsorted(grid, a), 1, 7)
    lo = up - 1
    dl, du = a - grid[lo], grid[up] - a
    code = np.where(dl < du, lo, np.where(du < dl, up, np.where(lo % 2 == 0, lo, up)))
    return (code | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def mx4_pack(codes):
    """Two codes a byte, the even column in the low half."""
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def mx4_quant(x):
    """(packed codes uint8 [T][C/2], scale bytes uint8 [T][C/32]) of x [T][C]."""
    x = np.asarray(x, dtype=np.float64)
    T, C = x.shape
    part = x.reshape(T, C // MX4_BLOCK, MX4_BLOCK)
    bad = ~np.isfinite(part).all(axis=2)
    amax = np.abs(np.where(np.isfinite(part), part, 0.0)).max(axis=2)
    k = np.where(amax > 0, np.frexp(amax)[1] - 3, 0)          # floor(log2) - 2
    k = np.maximum(k, -127)
    codes = e2m1_nearest(np.where(bad[..., None], 0.0, np.ldexp(np.where(bad[..., None], 0.0, part), -k[..., None])))
    scales = np.where(bad, 255, k + 127).astype(np.uint8)
    return mx4_pack(codes.reshape(T, C)), scales


def mx4_values(q, s):
    """float64 values [..][C] of packed codes [..][C/2] and scale bytes [..][C/32]."""
    codes = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return E2M1[codes] * np.repeat(scale, MX4_BLOCK, axis=-1)


def swiglu(y):
    """silu(even columns) * odd columns."""
    a, b = y[..., 0::2], y[..., 1::2]
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a)) * b


def mx4_moe(ids, weights, x, gate_up, down):
    """The layer's y [T][hidden] in float64, and the magnitudes its sums are of:
    ids, weights [T][k], x [T][hidden], gate_up [E][2 * inter][hidden] and down
    [E][hidden][inter] as values.  Returns (y, gu, gu_mag, h): per pair the
    gate/up sums, their magnitudes' sums and the activations."""
    T, k = ids.shape
    gu = np.zeros((T, k, gate_up.shape[1]))
    mag = np.zeros_like(gu)
    h = np.zeros((T, k, gate_up.shape[1] // 2))
    y = np.zeros((T, down.shape[1]))
    for t in range(T):
        for s in range(k):
            e = ids[t, s]
            if e < 0:
                continue
            gu[t, s] = gate_up[e] @ x[t]
            mag[t, s] = np.abs(gate_up[e]) @ np.abs(x[t])
            h[t, s] = swiglu(gu[t, s])
            y[t] += weights[t, s] * (down[e] @ h[t, s])
    return y, gu, mag, h
