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
