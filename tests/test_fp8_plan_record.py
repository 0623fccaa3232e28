"""The e4m3 product's table against the measured calls it was fitted to."""
import importlib.util
import os

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_tables_choices_are_near_the_best_measured_ones():
    spec = importlib.util.spec_from_file_location("fp8_plan_fit", os.path.join(ROOT, "profiles", "fp8_plan_fit.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    table, measured = fit.kernels(), fit.calls()
    assert len(table) == 12 and all(len(k.constants) == 7 for k in table)
    assert sum(len(v) for v in measured.values()) > 20000
    for what in ("exact-fp32", "exact-bf16", "fast-bf16"):
        part = fit.losses(table, {k: v for k, v in measured.items() if k[0] == what})
        assert np.mean([p[0] for p in part]) <= 1.02
        assert np.mean([p[0] for p in part if p[1] > 100]) <= 1.005
