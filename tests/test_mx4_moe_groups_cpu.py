"""The layer's launches are sized by the groups that its pairs can make: the
bound against every way to spread the pairs over the experts."""
import functools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "vq_dequant_matmul_gemv_amd", "csrc")


@pytest.fixture(scope="module")
def bound(tmp_path_factory):
    d = tmp_path_factory.mktemp("groups")
    (d / "m.cpp").write_text("""#include "vq_mx4_groups.h"
#include <cstdio>
int main() { for (int p, e, g; scanf("%d %d %d", &p, &e, &g) == 3;) printf("%d\\n", vqmi::mx4_moe_max_groups(p, e, g)); }
""")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "m.cpp"), "-o", str(d / "m")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        return [int(v) for v in subprocess.run([str(d / "m")], input=text, capture_output=True, text=True,
                                               check=True).stdout.split()]
    return run


@functools.lru_cache(None)
def most(pairs, experts, group):
    """Over every number of pairs that the last expert may have."""
    if pairs == 0 or experts == 0:
        return 0 if pairs == 0 else -10 ** 9
    return max(-(-c // group) + most(pairs - c, experts - 1, group) for c in range(pairs + 1))


def test_the_bound_is_reached_and_never_passed(bound):
    cases = [(p, e, g) for p in range(1, 33) for e in (1, 2, 3, 4, 5, 7, 8, 16, 31, 64) for g in (2, 4, 8)]
    assert bound(cases) == [most(*c) for c in cases]


def test_few_experts_make_more_groups_than_experts(bound):
    assert bound([(128, 8, 2), (128, 8, 4), (128, 2, 4), (1024, 1, 8), (8, 256, 2), (64, 64, 8)]) == [68, 38, 33, 128, 8, 64]


def test_the_launches_are_sized_by_it():
    text = open(os.path.join(CSRC, "vq_mx4_moe.hip")).read()
    run = text[text.index("void run_products"):]
    assert "mx4_moe_max_groups(a.pairs, a.experts, kGroup) * (tiles / MT)" in run[:run.index("\n}")]
