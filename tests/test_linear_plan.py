"""The linear layer's dispatch on the CPU: the sizes of linear_cases.py, which
the GPU tests run, reach every instantiation of its kernels. A changed rule
that moves a case to another kernel fails here."""
import itertools
import os
import shutil
import subprocess

import pytest

import linear_cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++")
ACTS = {"none": 0, "gelu": 1, "silu": 2}


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not CXX:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("plan") / "driver")
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "self_referential_memory_amd", "csrc", "layers"),
                    os.path.join(ROOT, "tests", "linear_plan_driver.cpp"), "-o", exe], check=True, timeout=120)

    def run(cases):
        """The instantiations that each case launches."""
        lines = [f"{M} {K} {N} {' '.join(str('fb'.index(c)) for c in t)} {ACTS[a]}" for M, K, N, t, a in cases]
        out = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, check=True, timeout=60)
        got = [line.split() for line in out.stdout.splitlines()]
        assert len(got) == len(lines)
        return got

    return run


def reached(plan, cases):
    return {name for names in plan(list(cases)) for name in names}


DENSE = ("BF16", "BF16_ANY", "FP32")
# two operands with rows of the same length are of one kind where both are bf16
SAME = [p for p in itertools.product(DENSE, repeat=2) if {"BF16", "BF16_ANY"} != set(p)]


def test_large_tiles_are_reached(plan):
    want = {"fwd_BF16_BF16_256", "gradx_BF16_BF16_256"} | {f"fwd_{a}_{b}_128" for a, b in SAME}
    want |= {f"{g}_{a}_{b}_128" for g in ("gradx", "gradw") for a, b in itertools.product(DENSE, repeat=2)}
    want |= {"slope", "splitw_128"}
    assert want <= reached(plan, linear_cases.large_tiles())


def test_small_tiles_are_reached(plan):
    want = {f"fwd_{a}_{b}_64" for a, b in SAME} | {"splitx_64", "splitw_64"}
    want |= {f"grads_{z}_{a}_{b}" for z in DENSE + ("SLOPE_BF16", "SLOPE_FP32") for a, b in SAME}
    assert want <= reached(plan, linear_cases.small_tiles())


def test_few_rows_are_reached(plan):
    want = set()
    for a, b in itertools.product(("FP32", "BF16"), repeat=2):
        shapes = ["1x1", "1x2", "2x2"]
        if (a, b) != ("FP32", "BF16"):
            shapes.append("2x1")
        if "FP32" in (a, b):
            shapes.append("2x4" if b == "BF16" else "4x2")
        want |= {f"few_{a}_{b}_{s}" for s in shapes}
    assert want <= reached(plan, linear_cases.few_rows())


def test_narrow_backward_is_reached(plan):
    """Every combination that the narrow form takes at all."""
    grid = [(66773, K, N, t, a) for K, N in itertools.product((64, 128, 256), repeat=2)
            for t in linear_cases.TYPES for a in ("none", "gelu")]
    want = {n for n in reached(plan, grid) if n.startswith("narrow")}
    assert len(want) > 60 and want <= reached(plan, linear_cases.narrow())
