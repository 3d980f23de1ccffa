"""The digits of the gated delta rule's fp32 results over whole sequences (the
states, the gradients of gates, strengths and states; with fp32 inputs all): what
fp32 sums lose and no more. Bounds and their derivation in delta_words."""
import pytest
import torch

from self_referential_memory_amd import srnl
from tests import delta_oracle, delta_words
from tests.delta_words import CASES, FINE, case_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_fp32_results(case, dtype):
    print("[delta digits]", case, dtype, flush=True)
    d, dout, dstate, eps, (out, S, grads) = case_inputs(case, dtype)
    x = {n: None if t is None else t.to(DEV) for n, t in d.items()}
    args = tuple(x[n] for n in ("q", "k", "v", "g", "beta"))
    o, S1, rec = srnl.gated_delta_fwd(*args, state=x["state"], norm_eps=eps, record=True)
    g = srnl.gated_delta_bwd(dout.to(DEV), *args, rec, state=x["state"], dstate=dstate.to(DEV), norm_eps=eps)
    lost = {"S": (delta_words.off(S1, S, 1), FINE[dtype]["out"])}
    if dtype == torch.float32:
        lost["out"] = delta_words.off(o, out, 2), FINE[dtype]["out"]
    for n, t in zip(("q", "k", "v", "g", "beta", "state"), g):
        if t.dtype == torch.float32:
            lost[n] = delta_words.off(t, grads[n], 1 if n == "state" else 2), FINE[dtype]["grad"]
    print({n: f"{e:.1e} of {b:.1e}" for n, (e, b) in lost.items()}, flush=True)
    assert all(e <= b for e, b in lost.values()), lost


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_chunks_that_last(dtype):
    """33 chunks under gates that keep e^-0.1 of a state over a chunk in the mean, so
    that what about ten chunks lose adds up, as independent errors do: the bounds times
    sqrt(10). (The reference is the rule token by token, as everywhere here.)"""
    B, T, Hk, H, Dk, Dv = 1, 2100, 1, 2, 32, 24
    d = delta_oracle.inputs(90, B, T, Hk, H, Dk, Dv, dtype, state=True, decay=0.005)
    gen = torch.Generator().manual_seed(91)
    dout = torch.randn((B, T, H, Dv), generator=gen).to(dtype)
    out, S, _, grads = delta_oracle.reference(d, norm_eps=1e-6, dout=dout)
    x = {n: None if t is None else t.to(DEV) for n, t in d.items()}
    args = tuple(x[n] for n in ("q", "k", "v", "g", "beta"))
    o, S1, rec = srnl.gated_delta_fwd(*args, state=x["state"], norm_eps=1e-6, record=True)
    g = srnl.gated_delta_bwd(dout.to(DEV), *args, rec, state=x["state"], norm_eps=1e-6)
    more = 10 ** 0.5
    lost = {"S": (delta_words.off(S1, S, 1), more * FINE[dtype]["out"]),
            "out": (delta_words.off(o, out, 2), more * FINE[dtype]["out"] + torch.finfo(dtype).eps / 2)}
    for n, t in zip(("q", "k", "v", "g", "beta", "state"), g):
        lost[n] = (delta_words.off(t, grads[n], 1 if n == "state" else 2),
                   more * FINE[dtype]["grad"] + (torch.finfo(t.dtype).eps / 2 if n in "qkv" else 0.0))
    print({n: f"{e:.1e} of {b:.1e}" for n, (e, b) in lost.items()}, flush=True)
    assert all(e <= b for e, b in lost.values()), lost
