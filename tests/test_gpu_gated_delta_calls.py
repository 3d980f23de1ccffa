"""Calls of the gated delta rule that a program may come to make without meaning
to, through every entry point."""
import pytest
import torch

from self_referential_memory_amd import srnl
from tests import delta_oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(B, T, seed=70):
    d = delta_oracle.inputs(seed, B, T, 2, 2, 16, 16, torch.float32, state=True)
    return {n: None if t is None else t.to(DEV) for n, t in d.items()}


@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("B,T", [(1, 5), (3, 1), (3, 5)])
def test_broadcast_inputs_are_refused(B, T, name):
    x = inputs(B, T)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    out, _, rec = srnl.gated_delta_fwd(*args, record=True)
    i = "qkv".index(name)
    args[i] = args[i][:1, :1].expand(args[i].shape)
    for call in (lambda: srnl.gated_delta_step(*args, x["state"]), lambda: srnl.gated_delta_fwd(*args),
                 lambda: srnl.gated_delta_bwd(out, *args, rec),
                 lambda: srnl.gated_delta(*args[:4], x["beta"].clone().requires_grad_())):
        with pytest.raises(ValueError, match=f"{name} must be contiguous"):
            call()
    args[i] = args[i].contiguous()
    assert srnl.gated_delta_fwd(*args)[0].isfinite().all()


def test_one_head_of_a_wider_row():
    x = inputs(3, 70)
    one = {n: t[:, :, :1].contiguous() if n != "state" else t[:, :1].contiguous() for n, t in x.items() if t is not None}
    wide = dict(one)
    for n in ("q", "k", "v"):
        p = torch.full((3, 70, 1, 40), float("nan"), device=DEV)
        p[..., 8:24] = one[n]
        wide[n] = p[..., 8:24]
    args, same = ([u[n] for n in ("q", "k", "v", "g", "beta")] for u in (one, wide))
    dout = torch.randn(3, 70, 1, 16, device=DEV)
    o, s, r = srnl.gated_delta_fwd(*args, record=True)
    o2, s2, r2 = srnl.gated_delta_fwd(*same, record=True)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    for a, b in zip(srnl.gated_delta_bwd(dout, *args, r)[:5], srnl.gated_delta_bwd(dout, *same, r2)[:5]):
        assert torch.equal(a, b)
    for a, b in zip(srnl.gated_delta_step(*args, one["state"].clone()), srnl.gated_delta_step(*same, one["state"].clone())):
        assert torch.equal(a, b)


def test_states_written_in_place_are_noticed_by_autograd():
    """A graph that holds the states from before an in-place call raises, as it does
    for torch's own in-place operations, and does not use what it finds there."""
    x = inputs(2, 5)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]

    def step():
        srnl.gated_delta_step(*args, x["state"])

    def forward():
        srnl.gated_delta_fwd(*args, state=x["state"], state_out=x["state"])

    for call in (step, forward):
        w = torch.ones_like(x["state"]).requires_grad_()
        loss = (w * x["state"]).sum()
        with torch.no_grad():
            call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        loss = (w * x["state"]).sum()
        with torch.no_grad():                     # into another tensor
            srnl.gated_delta_step(*args, x["state"], state_out=torch.empty_like(x["state"]))
        loss.backward()
        assert torch.equal(w.grad, x["state"])
    with torch.inference_mode():
        y = {n: t.clone() for n, t in x.items() if t is not None}
        srnl.gated_delta_step(*(y[n] for n in ("q", "k", "v", "g", "beta")), y["state"])


def test_a_step_without_states():
    """None: zeros before, none after."""
    x = inputs(2, 3)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    out, state = srnl.gated_delta_step(*args, None)
    want, _ = srnl.gated_delta_step(*args, torch.zeros_like(x["state"]))
    assert state is None and torch.equal(out, want)
