"""The 4-bit product's planner: what it chooses was measured, with weights from
memory, and is near the best; the replay that says so is the library's own loop."""
import importlib.util
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fit():
    spec = importlib.util.spec_from_file_location("mx4_plan_fit", os.path.join(ROOT, "profiles", "mx4_plan_fit.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    return fit


def test_every_choice_is_on_record_and_near_the_best(fit):
    """choices() goes through all candidates and raises where the one it ends
    with has no measured time."""
    table, (times, held) = fit.kernels(), fit.record()
    assert len(times) >= 1800 and len(held) == 300
    for x in ("mx4", "x16"):
        for pick, mean, worst in ((lambda key: key not in held, 1.01, 1.4), (lambda key: key in held, 1.015, 1.4)):
            part = {key: [(*q, t[0]) for q, t in runs.items()] for key, runs in times.items() if key[0] == x and pick(key)}
            loss = [p[0] for p in fit.losses(table, part)]
            assert np.mean(loss) <= mean and max(loss) <= worst


@pytest.mark.parametrize("x,T,rows,cols", [("mx4", 16, 8192, 8192), ("mx4", 24, 8192, 8192), ("mx4", 32, 8192, 8192),
                                           ("mx4", 16, 5120, 17408), ("mx4", 8, 17408, 5120), ("mx4", 32, 17408, 5120),
                                           ("x16", 8, 17408, 5120), ("x16", 16, 8192, 8192)])
def test_decode_shapes_with_cold_weights(fit, x, T, rows, cols):
    times, _ = fit.record()
    key = x, T, rows, cols
    loss = fit.losses(fit.kernels(), {key: [(*q, t[0]) for q, t in times[key].items()]})
    assert loss[0][0] <= 1.1


def test_the_library_makes_the_same_choices(fit):
    """The workspace of a shape's two plans, from the library and from the
    replay (choices closer than fp32 tells apart left out)."""
    from vq_dequant_matmul_gemv_amd import binding
    table, (times, _) = fit.kernels(), fit.record()
    checked = 0
    for T, rows, cols in sorted({key[1:] for key in times}):
        need, sure = 0, True
        for x in ("mx4", "x16"):
            options = fit.plans(table, (x, T, rows, cols))
            guess = fit.model([table[k].constants for k, _ in options],
                              [fit.features((x, T, rows, cols), table[k], s) for k, s in options])
            order = np.argsort(guess)
            sure = sure and (len(order) == 1 or guess[order[1]] > guess[order[0]] * (1 + 1e-5))
            s = options[order[0]][1]
            need = max(need, 4 * s * T * rows if s > 1 else 0)
        if sure:
            checked += 1
            assert binding.LIB.vq_mx4_workspace_bytes(rows, cols, T) == need, (T, rows, cols)
    assert checked > 1000
