"""The layers' corners, against their formulas in float64: operands shorter
than one wide load. Bounds as derived in test_gpu_layers.py."""
import pytest
import torch

from self_referential_memory_amd import srnl
from test_gpu_layers import BF16, F32, U, rnd, say, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x_t,w_t", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_linear_operands_shorter_than_a_load(x_t, w_t):
    """Every product whose operands have one to seven elements, and one side
    short while the other is not: a piece of eight is read elsewhere then, and
    counts as nothing."""
    say("short operands", x_t, w_t)
    for M, K, N in [(m, k, n) for k in range(1, 8) for m in (1, 2, 3, 7, 40) for n in (1, 2, 7, 33)]:
        x, w, b = rnd(M + K, M, K, dtype=x_t), rnd(N + K, N, K, dtype=w_t), rnd(3, N)
        X, W = x.double(), w.double()
        within(srnl.linear_fwd(x, w, b, out_dtype=F32), X @ W.t() + b.double(),
               2 * (K + 8) * U * (X.abs() @ W.abs().t() + b.double().abs()), f"{M} {K} {N}")
