"""The 4-bit product's table against the measured calls it was fitted to."""
import importlib.util
import os

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_tables_choices_are_near_the_best_measured_ones():
    spec = importlib.util.spec_from_file_location("mx4_plan_fit", os.path.join(ROOT, "profiles", "mx4_plan_fit.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    table, measured = fit.kernels(), fit.calls()
    assert len(table) == 24 and all(len(k.constants) == 7 for k in table)
    assert sum(len(v) for v in measured.values()) > 7000
    for x in ("mx4", "x16"):
        part = fit.losses(table, {k: v for k, v in measured.items() if k[0] == x})
        assert np.mean([p[0] for p in part]) <= 1.02
        assert np.mean([p[0] for p in part if p[1] > 20]) <= 1.01
    assert {c[0] for _, c, _ in fit.choices(table, measured)} == set(range(len(table)))  # every kernel is some call's
