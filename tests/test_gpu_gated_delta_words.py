"""The gated delta rule's bf16 outputs over whole sequences: what fp32 sums and
one rounding give, which values between products held in fewer bits would not.
Bounds and their derivation in delta_words."""
import pytest
import torch

from self_referential_memory_amd import srnl
from tests import delta_words
from tests.delta_words import CASES, case_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("case", CASES, ids=str)
def test_bf16_outputs_round_as_the_rule(case):
    print("[delta words]", case, flush=True)
    d, dout, dstate, eps, (out, S, grads) = case_inputs(case, torch.bfloat16)
    x = {n: None if t is None else t.to(DEV) for n, t in d.items()}
    args = tuple(x[n] for n in ("q", "k", "v", "g", "beta"))
    o, _, rec = srnl.gated_delta_fwd(*args, state=x["state"], norm_eps=eps, record=True)
    g = srnl.gated_delta_bwd(dout.to(DEV), *args, rec, state=x["state"], dstate=dstate.to(DEV), norm_eps=eps)
    off = {}
    for n, t, ref in (("out", o, out), ("q", g[0], grads["q"]), ("k", g[1], grads["k"]), ("v", g[2], grads["v"])):
        off[n] = delta_words.on_other_sides(t, ref, delta_words.TOL[n])
    print(off, flush=True)
    assert all(count <= most for count, most in off.values()), off
