"""Every instantiation of the linear layer's kernels (linear_cases.py; that the
cases reach them is held on the CPU by test_linear_plan.py), forward and
backward, against float64 with the bounds of test_gpu_layers.py."""
import pytest

import linear_cases
from test_gpu_layers import BF16, F32, check_linear

pytestmark = pytest.mark.gpu
T = {"f": F32, "b": BF16}


def run(cases, types=None):
    for i, (M, K, N, t, act) in enumerate(cases):
        if types is None or t == types:
            x, w, y = (T[c] for c in t)
            check_linear(M, K, N, x, w, y, act=act, bias=i % 3 > 0, res=y if i % 4 == 1 else None,
                         add=i % 5 > 2, seed=7 + i)


@pytest.mark.parametrize("types", linear_cases.TYPES, ids="".join)
@pytest.mark.parametrize("family", ["large_tiles", "small_tiles", "narrow"])
def test_linear_dispatch(family, types):
    run(getattr(linear_cases, family)(), types)


def test_linear_dispatch_few_rows():
    run(linear_cases.few_rows())
