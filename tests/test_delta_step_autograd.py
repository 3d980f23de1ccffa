"""gated_delta_step has no gradient: where autograd would need one it raises,
before any work and before it writes a state. On the CPU."""
import pytest
import torch
from torch.autograd import forward_ad

from self_referential_memory_amd import srnl


def args():
    q, v, w = torch.randn(2, 3, 1, 16), torch.randn(2, 3, 2, 24), torch.rand(2, 3, 2)
    return [q, q.clone(), v, -w, w, torch.randn(2, 2, 16, 24)]


@pytest.mark.parametrize("i", range(6))
def test_a_wanted_gradient_raises(i):
    a = args()
    a[i].requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient"):
        srnl.gated_delta_step(*a)
    with pytest.raises(RuntimeError, match="no gradient"):
        srnl.gated_delta_step(*a, state_out=torch.empty(2, 2, 16, 24))
    # a tracked intermediate, as a projection's slice is
    a = args()
    leaf = a[i].clone().requires_grad_()
    a[i] = leaf * 2
    with pytest.raises(RuntimeError, match="no gradient"):
        srnl.gated_delta_step(*a)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):       # as far as a CPU tensor goes
        srnl.gated_delta_step(*a)
    a[i] = a[i].detach()
    with pytest.raises(ValueError, match="GPU"):
        srnl.gated_delta_step(*a)


@pytest.mark.parametrize("i", range(6))
def test_a_tangent_raises(i):
    a = args()
    with forward_ad.dual_level():
        a[i] = forward_ad.make_dual(a[i], torch.ones_like(a[i]))
        with pytest.raises(RuntimeError, match="no gradient"):
            srnl.gated_delta_step(*a)


def test_a_tracked_buffer_raises():
    a = args()
    for kw in ({"state_out": torch.empty(2, 2, 16, 24)}, {"out": torch.empty(2, 3, 2, 24)}):
        next(iter(kw.values())).requires_grad_()
        with pytest.raises(RuntimeError, match="no gradient"):
            srnl.gated_delta_step(*a, **kw)


def test_no_states_at_all():
    a = args()
    with pytest.raises(ValueError, match="GPU"):
        srnl.gated_delta_step(*a[:5], None)
    a[0].requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient"):
        srnl.gated_delta_step(*a[:5], None)
