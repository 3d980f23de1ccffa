"""The layers' autograd nodes without a GPU: the library's calls replaced by
stand-ins, to see which calls autograd is told of."""
import pytest
import torch
from torch.autograd import forward_ad

from self_referential_memory_amd import srnl


@pytest.fixture
def calls(monkeypatch):
    """Every forward entry point returns zeros of its output's shape."""
    def norm(x, gain, bias, eps=1e-5, *, out_dtype=None, stats=False, **kw):
        y = torch.zeros(x.shape)
        return (y, torch.zeros(x.shape[:-1]), torch.ones(x.shape[:-1])) if stats else y

    def lin(x, w, bias=None, *, keep_pre=False, **kw):
        y = torch.zeros(x.shape[:-1] + w.shape[:1])
        return (y, y.clone()) if keep_pre else y

    monkeypatch.setattr(srnl, "layer_norm_fwd", norm)
    monkeypatch.setattr(srnl, "linear_fwd", lin)
    monkeypatch.setattr(srnl, "dwconv_fwd", lambda u, *a, **kw: torch.zeros(u.shape))
    x, g = torch.randn(4, 8), torch.randn(8)
    w, b, r = torch.randn(6, 8), torch.randn(6), torch.randn(4, 6)
    u, cw, a = torch.randn(1, 2, 2, 8), torch.randn(8, 3, 3), torch.randn(1, 2, 2, 8)
    return {"layer_norm": (srnl.layer_norm, [x, g, g.clone()]),
            "linear": (lambda *t: srnl.linear(*t[:3], act="gelu", residual=t[3]), [x, w, b, r]),
            "dwconv": (srnl.dwconv, [u, cw, g, a, a.clone()])}


@pytest.mark.parametrize("op", ["layer_norm", "linear", "dwconv"])
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(calls, op, grad):
    """A tangent on any input raises, as in srnl.operator; it is not lost."""
    f, args = calls[op]
    for i in range(len(args)):
        with torch.set_grad_enabled(grad), forward_ad.dual_level():
            dual = list(args)
            dual[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(RuntimeError, match="jvp"):
                f(*dual)
            f(*args)                        # no tangent: an ordinary call


@pytest.mark.parametrize("op", ["layer_norm", "linear", "dwconv"])
def test_reverse_mode_nodes_only_where_wanted(calls, op):
    f, args = calls[op]
    assert f(*args).grad_fn is None
    for i in range(len(args)):
        leaf = [t.clone().requires_grad_(j == i) for j, t in enumerate(args)]
        assert f(*leaf).grad_fn is not None
        with torch.no_grad():
            assert f(*leaf).grad_fn is None
