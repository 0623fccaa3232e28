"""The time model behind the 4-bit product's choice of kernel and splits.

    python3 profiles/mx4_plan_fit.py            # what the table's choices lose against the best measured ones
    python3 profiles/mx4_plan_fit.py --fit      # the constants fitted anew, and what their choices lose

Reads the measured calls (mx4_product_calls.txt beside this file) and the table `kMx4Kernels` in csrc/vq_mx4.hip.
A call's time is that of the calls captured into one graph, the median of three replays, with bf16 y: the geometric
mean of one over weights that rotate through 400 MB (64 weights at most) and of one over two weights in turn.
"""

import collections
import os
import re
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(HERE, "..", "vq_dequant_matmul_gemv_amd", "csrc", "vq_mx4.hip")
CALLS = os.path.join(HERE, "mx4_product_calls.txt")

Kernel = collections.namedtuple("Kernel", "rows tokens k_waves unit mx4 constants")
LOW = [1, 0, .02, 2, .05, 0, 0]      # bounds of base, latency, rate, bw, join, unit, x_share
HIGH = [12, 3, 3, 8, 2, 8, 1.2]
STARTS = ([4, 1, .5, 4, .2, .1, .1], [4, .3, .1, 4, .3, .5, .5], [5, .5, .2, 4, .3, .1, .1], [8, 1, 1, 6, .2, 3, 1])


def kernels():
    """The table's rows: tile, waves (or groups of them) that split the columns, blocks that splits are multiples of,
    4-bit x or 16-bit, the model's seven constants."""
    text = open(SOURCE).read()
    text = text[text.index("const Mx4Kernel kMx4Kernels[] = {"):]
    rows = re.findall(r"\{(\d+), (\d+), (\d+), (\d+), (true|false), ([^}]*), run_", text[:text.index("\n};")])
    return [Kernel(int(r), int(t), int(w), int(u), m == "true", np.array([float(c.rstrip("f")) for c in rest.split(", ")]))
            for r, t, w, u, m, rest in rows]


def calls():
    """{(x, T, rows, cols): [(kernel, splits, us), ...]}; x: "mx4" or "x16"."""
    out = {}
    for line in open(CALLS):
        if line.startswith("#"):
            continue
        key, times = line.split(" : ")
        x, T, rows, cols = key.split()
        out[x, int(T), int(rows), int(cols)] = [
            (int(a), int(b), float(c)) for a, b, c in re.findall(r"(\d+)/(\d+)=([\d.]+)", times)]
    return out


def features(key, kernel, splits):
    """What the model takes of a call: T, rows, blocks of 32 columns, splits, blocks a split, work units, tile rows,
    k_waves, bytes of a token's block."""
    x, T, rows, cols = key
    blocks = cols // 32
    part = -(-(-(-blocks // splits)) // kernel.unit) * kernel.unit
    units = -(-rows // kernel.rows) * -(-T // kernel.tokens) * splits
    return (T, rows, blocks, splits, part, units, kernel.rows, kernel.k_waves, 17 if x == "mx4" else 64)


def model(constants, f):
    """plan_time of csrc/vq_mx4.hip, over an array of features."""
    T, rows, blocks, splits, part, units, tile_rows, k_waves, x_bytes = np.asarray(f, dtype=float).T
    base, latency, rate, bw, join, unit, x_share = np.abs(constants)
    steps = .25 * part / k_waves
    serial = latency * np.ceil(steps)
    load = np.ceil(units / 256) * (rate * steps + unit)
    mem = (17 * rows * blocks + 4 * T * rows + x_share * x_bytes * T * blocks * rows / tile_rows) * 1e-6 / bw
    return base + (serial ** 4 + load ** 4 + mem ** 4) ** .25 + np.where(splits > 1, 2 + join * splits * T * rows * 8e-6, 0)


def choices(table, measured):
    """[(key, the call chosen, the best call)] of the model's choices among the measured calls."""
    out = []
    for key, runs in measured.items():
        guess = [model(table[k].constants, [features(key, table[k], s)])[0] for k, s, _ in runs]
        out.append((key, runs[int(np.argmin(guess))], min(runs, key=lambda r: r[2])))
    return out


def losses(table, measured):
    """[(chosen call's time / best call's, best time, key)]."""
    return [(c[2] / b[2], b[2], key) for key, c, b in choices(table, measured)]


def report(table, measured):
    for x in sorted({key[0] for key in measured}):
        part = losses(table, {k: v for k, v in measured.items() if k[0] == x})
        r, big = np.array([p[0] for p in part]), np.array([p[0] for p in part if p[1] > 20])
        print(f"{x}: {len(part)} shapes, mean {r.mean():.4f}, 90 % below {np.quantile(r, .9):.3f}, worst {r.max():.2f}; "
              f"above 20 us: {len(big)}, mean {big.mean():.4f}")


def fit(table, measured, rounds=40):
    """The table with constants fitted to the calls, the faster ones of a shape weighing more; after each round the
    calls of wrong choices gain weight, and the round with the least loss stays."""
    from scipy.optimize import least_squares
    more = collections.Counter()

    def row(k, starts):
        f, us, weight = [], [], []
        for key, runs in measured.items():
            best = min(r[2] for r in runs)
            for a, s, t in runs:
                if a == k:
                    f.append(features(key, table[k], s))
                    us.append(t)
                    weight.append((best / t) ** 2 * np.exp(more[key, a, s]))
        f, us, weight = np.array(f, dtype=float), np.array(us), np.array(weight)
        runs = [least_squares(lambda p: weight * np.log(model(p, f) / us), np.clip(x0, LOW, HIGH), bounds=(LOW, HIGH),
                              loss="soft_l1", f_scale=.1) for x0 in starts]
        return table[k]._replace(constants=min(runs, key=lambda r: r.cost).x)

    now, best = [row(k, STARTS) for k in range(len(table))], None
    for _ in range(rounds):
        chosen = choices(now, measured)
        loss = np.array([c[2] / b[2] for _, c, b in chosen])
        cost = np.log(loss).mean() + np.maximum(loss - 1.05, 0).mean()
        if best is None or cost < best[0]:
            best = cost, now
        for key, c, b in chosen:
            if c[2] > 1.03 * b[2]:
                gain = np.log(min(1 + 3 * (c[2] / b[2] - 1), 2))
                more[(key, *c[:2])] += gain
                more[(key, *b[:2])] += min(gain, np.log(1.5))
        now = [row(k, [now[k].constants]) for k in range(len(table))]
    for k, kernel in enumerate(best[1]):
        print(k, kernel[:4], ", ".join(f"{c:.3g}f" for c in kernel.constants))
    return best[1]


if __name__ == "__main__":
    now, seen = kernels(), calls()
    report(fit(now, seen) if "--fit" in sys.argv[1:] else now, seen)
