"""The plan of the fused grouped products (csrc/group_plan.h) for the shapes of
tests/group_cases.py, and its limits over all shapes."""
import os
import random
import shutil
import subprocess

import pytest

from group_cases import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "group_plan")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "nf4_base_lora_b200", "csrc"), os.path.join(ROOT, "tests", "c", "group_plan.cc"),
                    "-o", exe], check=True)

    def ask(shapes):
        text = "".join("%d %d %d %d %d %d\n" % s for s in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


@pytest.mark.parametrize("name", CASES)
def test_the_cases_take_the_paths_that_they_are_for(plans, name):
    E, N, K, r, rows, fwd, dx = CASES[name]
    M = sum(rows)
    for want, (tile, tile_rows, splits, steps, pairs), cols in zip(
            (fwd, dx), plans([(0, E or 1, M, N, K, r), (1, E or 1, M, K, N, r)]), (N, K)):
        if want is None:
            continue
        tiles = sum(-(-n // tile_rows) for n in rows) * -(-cols // 256) * splits
        assert (tile, splits > 1) == want[:2], (tile, splits)
        assert not want[2] or tiles > pairs, tiles
        assert steps >= want[3], steps


def test_every_fused_kernel_is_covered_both_ways():
    for kind in (5, 6):
        walked = {c[kind][0] for c in CASES.values() if c[kind] and c[kind][2]}
        split = {c[kind][0] for c in CASES.values() if c[kind] and c[kind][1]}
        assert walked == split == {64 if kind == 5 else 32, 256, 512}


def test_plans_stay_within_the_kernels_limits(plans):
    rng = random.Random(3)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    shapes = [(rng.randrange(2), log(1, 4096), log(1, 1 << 24), 8 * log(1, 1 << 13), 8 * log(1, 1 << 13),
               log(1, 256)) for _ in range(20000)]
    for (dx, E, M, cols, contraction, r), (tile, rows, splits, steps, _) in zip(shapes, plans(shapes)):
        assert tile in (32 if dx else 64, 256, 512) and 32 <= rows <= tile and rows % 32 == 0
        wide = 64 if tile == 512 else 128
        assert steps == -(-contraction // wide)
        assert splits == 1 or (2 <= splits <= 8 and 4 * splits <= steps)
