"""The time model behind the e4m3 product's choice of kernel and splits.

    python3 profiles/fp8_plan_fit.py            # what the table's choices lose against the best measured ones
    python3 profiles/fp8_plan_fit.py --fit      # the constants fitted anew, and what their choices lose

Reads the measured calls (fp8_product_calls.txt beside this file) and the table `kFp8Kernels` in csrc/vq_fp8.hip.
A call's time is that of six calls captured into one graph, the median of two replays, over weights that rotate
through 600 MB.
"""

import collections
import os
import re
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(HERE, "..", "vq_dequant_matmul_gemv_amd", "csrc", "vq_fp8.hip")
CALLS = os.path.join(HERE, "fp8_product_calls.txt")

Kernel = collections.namedtuple("Kernel", "rows tokens k_waves constants")
LOW = [1, 0, .05, 2, .05, 0, 0]      # bounds of base, latency, rate, bw, join, unit, x_share
HIGH = [12, 3, 3, 8, 2, 8, 1.2]
STARTS = ([4, 1, .5, 4, .2, .1, .1], [4, 1, .3, 4, .3, .5, .5], [5, .5, .2, 4, .3, .1, .1], [8, 1, 1, 6, .2, 3, 1])


def kernels():
    """The table's rows: tile, waves that split the columns, the model's seven constants."""
    text = open(SOURCE).read()
    text = text[text.index("const Fp8Kernel kFp8Kernels[] = {"):]
    rows = re.findall(r"\{(\d+), (\d+), (\d+), \d+, \w+, (?:true|false), (?:true|false),([^}]*)\}",
                      text[:text.index("\n};")])
    return [Kernel(int(r), int(t), int(w), np.array([float(c) for c in re.findall(r"([\d.]+)f\b", rest)]))
            for r, t, w, rest in rows]


def calls():
    """{(products, T, rows, cols): [(kernel, splits, us), ...]}; products: exact with an fp32 or a bf16 y, or fast."""
    out = {}
    for line in open(CALLS):
        if line.startswith("#"):
            continue
        key, times = line.split(" : ")
        what, T, rows, cols = key.split()
        out[what, int(T), int(rows), int(cols)] = [
            (int(a), int(b), float(c)) for a, b, c in re.findall(r"(\d+)/(\d+)=([\d.]+)", times)]
    return out


def features(key, kernel, splits):
    """What the model takes of a call: T, rows, cols, splits, column blocks a split, blocks, tile rows, k_waves."""
    _, T, rows, cols = key
    kb, whole = -(-cols // 128), 1 if kernel.k_waves > 1 else 4
    steps = -(-(-(-kb // splits)) // whole) * whole
    return (T, rows, cols, splits, steps, -(-rows // kernel.rows) * -(-T // kernel.tokens) * splits, kernel.rows,
            kernel.k_waves)


def model(constants, f):
    """plan_time of csrc/vq_fp8.hip, over an array of features."""
    T, rows, cols, splits, steps, units, tile_rows, k_waves = np.asarray(f, dtype=float).T
    base, latency, rate, bw, join, unit, x_share = np.abs(constants)
    serial = latency * np.ceil(steps / k_waves)
    load = np.ceil(units / 256) * (rate * steps / k_waves + unit)
    mem = (rows * cols + 4 * T * rows + x_share * T * cols * rows / tile_rows) * 1e-6 / bw
    return base + (serial ** 4 + load ** 4 + mem ** 4) ** .25 + np.where(splits > 1, 2 + join * splits * T * rows * 8e-6, 0)


def losses(table, measured):
    """[(chosen call's time / best call's, best time, key)] of the model's choices among the measured calls."""
    out = []
    for key, runs in measured.items():
        guess = [model(table[k].constants, [features(key, table[k], s)])[0] for k, s, _ in runs]
        best = min(us for _, _, us in runs)
        out.append((runs[int(np.argmin(guess))][2] / best, best, key))
    return out


def report(table, measured):
    for what in sorted({key[0] for key in measured}):
        part = losses(table, {k: v for k, v in measured.items() if k[0] == what})
        r, big = np.array([p[0] for p in part]), np.array([p[0] for p in part if p[1] > 100])
        print(f"{what}: {len(part)} shapes, mean {r.mean():.4f}, 90 % below {np.quantile(r, .9):.3f}, worst {r.max():.2f}; "
              f"above 100 us: {len(big)}, mean {big.mean():.4f}")


def fit(table, measured):
    """The table with constants fitted to the calls it was fitted to, the faster ones of a shape weighing more."""
    from scipy.optimize import least_squares
    rows = collections.defaultdict(list)
    for key, runs in measured.items():
        if key[0] == "exact-bf16":
            continue                       # measured later, with the table as it is
        best = min(us for _, _, us in runs)
        for k, s, us in runs:
            rows[k].append((*features(key, table[k], s), us, (best / us) ** 2))
    out = []
    for k, kernel in enumerate(table):
        a = np.array(rows[k])
        f, us, weight = a[:, :8], a[:, 8], a[:, 9]
        runs = [least_squares(lambda p: weight * np.log(model(p, f) / us),
                              np.clip(x0, np.array(LOW) + 1e-3, np.array(HIGH) - 1e-3), bounds=(LOW, HIGH))
                for x0 in STARTS]
        x = min(runs, key=lambda r: r.cost).x
        print(k, kernel[:3], f"{len(a)} calls", ", ".join(f"{c:.3f}f" for c in x),
              f"rms {np.log(model(x, f) / us).std():.3f}")
        out.append(kernel._replace(constants=x))
    return out


if __name__ == "__main__":
    now, seen = kernels(), calls()
    report(fit(now, seen) if "--fit" in sys.argv[1:] else now, seen)
