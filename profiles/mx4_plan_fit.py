"""The time model behind the 4-bit product's choice of kernel and splits.

    python3 profiles/mx4_plan_fit.py            # what the table's choices lose against the best measured calls
    python3 profiles/mx4_plan_fit.py --fit      # the constants fitted anew, and what their choices lose

Reads the measured calls (mx4_product_calls.txt beside this file) and the table `kMx4Kernels` with `kMx4Split` and
`kMx4Splits` in csrc/vq_mx4.hip, and goes through the same candidates as `make_plan` there: a choice that nobody measured
is an error.  A shape has the times of its calls captured into one graph with bf16 y, each the median of three replays:
"cold" over weights at distinct places, read once a replay after 640 MB of other data were read, and "warm" over two
weights in turn.  A pass through a model's layers meets the cold ones.  Shapes marked as held out or later are not fitted.
"""

import collections
import os
import re
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(HERE, "..", "vq_dequant_matmul_gemv_amd", "csrc", "vq_mx4.hip")
CALLS = os.path.join(HERE, "mx4_product_calls.txt")
PLANES = 512 << 20                   # kMaxPlanBytes: fp32 planes of a split

Kernel = collections.namedtuple("Kernel", "rows tokens k_waves unit mx4 constants")


def kernels():
    """The table's rows: tile, waves (or groups of them) that split the columns, blocks that splits are multiples of,
    4-bit x or 16-bit, the model's seven constants."""
    text = open(SOURCE).read()
    text = text[text.index("const Mx4Kernel kMx4Kernels[] = {"):]
    rows = re.findall(r"\{(\d+), (\d+), (\d+), (\d+), (true|false), ([^}]*), run_", text[:text.index("\n};")])
    return [Kernel(int(r), int(t), int(w), int(u), m == "true", np.array([float(c.rstrip("f")) for c in rest.split(", ")]))
            for r, t, w, u, m, rest in rows]


def split_cost():
    """us of the launch that joins a split's planes."""
    return float(re.search(r"constexpr float kMx4Split = ([\d.]+)f;", open(SOURCE).read()).group(1))


def split_counts():
    """The numbers of splits that a plan may have."""
    return [int(s) for s in re.search(r"constexpr int kMx4Splits\[\] = \{([\d, ]+)\};", open(SOURCE).read()).group(1).split(",")]


def record(later=False):
    """{(x, T, rows, cols): {(kernel, splits): (cold us, warm us)}} and the shapes that are not fitted; x: "mx4" or "x16".
    later: with those that were measured after the fit."""
    out, held, hold = {}, set(), False
    for line in open(CALLS):
        if line.startswith("# later") and not later:
            break
        if line.startswith("#"):
            hold = hold or line.startswith("# held out")
            continue
        key, times = line.split(" : ")
        x, T, rows, cols = key.split()
        key = x, int(T), int(rows), int(cols)
        out[key] = {(int(a), int(b)): (float(c), float(w))
                    for a, b, c, w in re.findall(r"(\d+)/(\d+)=([\d.]+),([\d.]+)", times)}
        if hold:
            held.add(key)
    return out, held


def calls():
    """{(x, T, rows, cols): [(kernel, splits, cold us), ...]}."""
    return {key: [(k, s, t[0]) for (k, s), t in runs.items()] for key, runs in record()[0].items()}


def plans(table, key):
    """[(kernel, splits)] that make_plan compares for a shape."""
    x, T, rows, cols = key
    out = []
    for i, k in enumerate(table):
        if k.mx4 != (x == "mx4") or -(-rows // k.rows) * -(-T // k.tokens) >= 1 << 22:
            continue
        for s in split_counts():
            part = -(-(-(-cols // 32 // s)) // k.unit) * k.unit
            if -(-cols // 32 // part) == s and (s == 1 or s * T * rows * 4 <= PLANES):
                out.append((i, s))
    return out


def features(key, kernel, splits):
    """What the model takes of a call: T, rows, blocks of 32 columns, splits, blocks a split, work units, row tiles,
    k_waves, bytes of a token's block."""
    x, T, rows, cols = key
    blocks = cols // 32
    part = -(-(-(-blocks // splits)) // kernel.unit) * kernel.unit
    row_tiles = -(-rows // kernel.rows)
    return (T, rows, blocks, splits, part, row_tiles * -(-T // kernel.tokens) * splits, row_tiles, kernel.k_waves,
            17 if x == "mx4" else 64)


def model(constants, f, split=None):
    """plan_time of csrc/vq_mx4.hip, over an array of features; constants: seven, or seven for each row of f."""
    T, rows, blocks, splits, part, units, row_tiles, k_waves, x_bytes = np.asarray(f, dtype=float).T
    base, latency, rate, bw, join, unit, x_share = np.asarray(constants).T
    steps = .25 * part / k_waves
    serial = latency * np.ceil(steps)
    load = np.ceil(units / 256) * (rate * steps + unit)
    mem = (17 * rows * blocks + 4 * T * rows + (1 + x_share * (row_tiles - 1)) * x_bytes * T * blocks) * 1e-6 / bw
    joining = np.where(splits > 1, (split_cost() if split is None else split) + join * splits * T * rows * 8e-6, 0)
    return base + (serial ** 4 + load ** 4 + mem ** 4) ** .25 + joining


def choices(table, measured, split=None):
    """[(key, the call that make_plan chooses, the best call)], calls as in `measured` (kernel, splits, us)."""
    out = []
    for key, runs in measured.items():
        options = plans(table, key)
        guess = model([table[k].constants for k, _ in options], [features(key, table[k], s) for k, s in options], split)
        chosen = options[int(np.argmin(guess))]
        found = [r for r in runs if tuple(r[:2]) == chosen]
        if not found:
            raise LookupError(f"{key}: the choice {chosen} is not on record")
        out.append((key, found[0], min(runs, key=lambda r: r[2])))
    return out


def losses(table, measured, split=None):
    """[(chosen call's time / best call's, best time, key)]."""
    return [(c[2] / b[2], b[2], key) for key, c, b in choices(table, measured, split)]


def report(table, split=None):
    times, held = record(later=True)
    for x in ("mx4", "x16"):
        for name, pick in (("fitted", lambda key: key not in held), ("held out", lambda key: key in held)):
            for k, state in enumerate(("cold", "warm")):
                part = {key: [(*q, t[k]) for q, t in runs.items()] for key, runs in times.items() if key[0] == x and pick(key)}
                if state == "warm":    # of the same choices
                    chosen = {key: c[:2] for key, c, _ in choices(table, part, split)}
                    loss = [(times[key][chosen[key]][1] / min(t[1] for t in times[key].values()), 0) for key in part]
                else:
                    loss = losses(table, part, split)
                r, big = np.array([p[0] for p in loss]), np.array([p[0] for p in loss if p[1] > 20])
                print(f"{x}, {name}, {state}: {len(loss)} shapes, mean {r.mean():.4f}, 95 % below {np.quantile(r, .95):.3f}, "
                      f"worst {r.max():.2f}" + (f"; above 20 us: {len(big)}, mean {big.mean():.4f}" if len(big) else ""))


def fit(table, steps=5000, fidelity=.03, warm=.5, heavy=4.):
    """The table and the split's cost with the least loss of the choices: gradients of the loss that each shape expects
    when calls are taken with the softmax of their predicted times, which sharpens from 12 to 1.5 %, and `fidelity` of the
    predictions' own errors.  A call's loss is that of its cold time, what is above 5 % of it four times, and `warm` of
    that of its warm one, which decides between calls that take nearly the same time with cold weights.  Weights of 2^24
    values and more count `heavy` times; calls that are not on record (twice the best and more) as 4 times the best."""
    import torch
    times, held = record()
    keys = [key for key in times if key not in held]
    options = [plans(table, key) for key in keys]
    flat = [(i, k, s) for i, part in enumerate(options) for k, s in part]
    shape = torch.tensor([i for i, _, _ in flat])
    kernel = torch.tensor([k for _, k, _ in flat])
    f = torch.tensor(np.array([features(keys[i], table[k], s) for i, k, s in flat], dtype=float))
    best = [min(t[0] for t in times[key].values()) for key in keys]
    us = torch.tensor([times[keys[i]].get((k, s), (4 * best[i], 0))[0] for i, k, s in flat], dtype=torch.float64)
    cost = torch.log(us / torch.tensor(best, dtype=torch.float64)[shape])
    seen = cost < .69
    warmest = [min(t[1] for t in times[key].values()) for key in keys]
    second = torch.tensor([np.log(times[keys[i]].get((k, s), (0, 4 * warmest[i]))[1] / warmest[i]) for i, k, s in flat])
    weight = torch.tensor([heavy if key[2] * key[3] >= 1 << 24 else 1. for key in keys], dtype=torch.float64)
    value = (cost + 3 * torch.relu(cost - .05) + warm * second) * (weight / weight.mean())[shape]
    T, rows, blocks, splits, part, units, row_tiles, k_waves, x_bytes = f.T
    wave_steps, rounds, is_split = .25 * part / k_waves, torch.ceil(units / 256), (splits > 1).double()
    raw = torch.tensor(np.log(np.maximum([k.constants for k in table], 2e-3))).requires_grad_(True)
    split = torch.tensor(np.log(split_cost())).requires_grad_(True)

    def predict():
        base, latency, rate, bw, join, unit, share = torch.exp(raw)[kernel].T
        mem = (17 * rows * blocks + 4 * T * rows + (1 + share * (row_tiles - 1)) * x_bytes * T * blocks) * 1e-6 / bw
        four = (latency * torch.ceil(wave_steps)) ** 4 + (rounds * (rate * wave_steps + unit)) ** 4 + mem ** 4
        return base + (four + 1e-12) ** .25 + is_split * (torch.exp(split) + join * splits * T * rows * 8e-6)

    def over(values, how, empty):
        return torch.full((len(keys),), empty, dtype=torch.float64).scatter_reduce(0, shape, values, how)

    optimizer, kept = torch.optim.Adam([raw, split]), (np.inf, None, None)
    for step in range(steps):
        late = step / steps
        for group in optimizer.param_groups:
            group["lr"] = .012 * (1 - late) + .001
        guess = torch.log(predict())
        z = -guess / (.12 * (1 - late) + .015 * late)
        e = torch.exp(z - over(z.detach(), "amax", -1e9)[shape])
        share = e / over(e, "sum", 0.)[shape]
        expected = over(share * value, "sum", 0.).mean()
        loss = expected + fidelity * (guess - torch.log(us))[seen].abs().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        with torch.no_grad():
            raw.clamp_(np.log(1e-3), np.log(12.))
            if step % 20 == 0 or step == steps - 1:
                guess = torch.log(predict())
                chosen = guess <= over(guess, "amin", 1e9)[shape]
                hard = over(torch.where(chosen, value, torch.zeros_like(value)), "amax", 0.).mean().item()
                unused = len(table) - len(set(kernel[chosen].tolist()))
                if hard + .001 * unused < kept[0]:
                    kept = hard + .001 * unused, torch.exp(raw).numpy().copy(), torch.exp(split).item()
        if step % 400 == 0:
            print(step, f"expected {expected.item():.4f}, chosen {hard:.4f}, unused {unused}", flush=True)
    rounded = [np.array([float(f"{v:.3g}") if v > 2e-3 else 0. for v in row]) for row in kept[1]]
    new, split = [k._replace(constants=c) for k, c in zip(table, rounded)], float(f"{kept[2]:.3g}")
    for k in new:
        print("{" + f"{k.rows}, {k.tokens}, {k.k_waves}, {k.unit}, {str(k.mx4).lower()}, "
              + ", ".join(f"{v:g}" + ("f" if v != int(v) else "") for v in k.constants) + ", ...},")
    print("kMx4Split", split)
    return new, split


if __name__ == "__main__":
    now, cost = kernels(), split_cost()
    report(*(fit(now) if "--fit" in sys.argv[1:] else (now, cost)))
