"""The layers' refusals, on the CPU: invalid sizes, types and pointers return
their status before any device work, and the binding checks shapes first."""
import ctypes

import pytest
import torch

from self_referential_memory_amd import srnl

ARG, DTYPE, PTR, WS, OK = (srnl.SRNL_ERR_ARG, srnl.SRNL_ERR_DTYPE, srnl.SRNL_ERR_PTR,
                           srnl.SRNL_ERR_WORKSPACE, srnl.SRNL_OK)


def norm_fwd(x=0, rows=2, C=8, i=0, o=0, eps=1e-5):
    return srnl.lib().srnl_layer_norm_fwd(x, rows, C, i, None, None, eps, o, None, None, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), ARG), (dict(C=0), ARG), (dict(C=-8), ARG), (dict(rows=1 << 62, C=1 << 20), ARG),
    (dict(C=(1 << 30) + 8), ARG), (dict(C=(1 << 31) - 1), ARG),
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(i=2), DTYPE), (dict(o=-1), DTYPE), (dict(), PTR),
    (dict(x=24), PTR), (dict(rows=0), OK)])
def test_norm_forward_errors(kw, status):
    assert norm_fwd(**kw) == status
    assert (srnl.lib().srnl_last_error().decode() == "") == (status == OK)


def norm_bwd(rows=2, C=8, i=0, o=0, add=None, add_t=0, dgain=None, ws=None, nws=0):
    return srnl.lib().srnl_layer_norm_bwd(None, o, None, rows, C, i, None, None, None, add, add_t,
                                          None, dgain, None, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), ARG), (dict(C=0), ARG), (dict(i=9), DTYPE), (dict(add=16, add_t=5), DTYPE),
    (dict(rows=999, dgain=16), WS), (dict(rows=999, dgain=16, ws=16, nws=8), WS), (dict(), PTR), (dict(rows=0), OK)])
def test_norm_backward_errors(kw, status):
    assert norm_bwd(**kw) == status


def linear(fn, M=2, K=8, N=8, act=0, types=(0, 0, 0, 0), res=None, params=True, dw=None, db=None):
    p = srnl.LinearParams(None, None, res, *types, act, None)
    pp = ctypes.byref(p) if params else None
    if fn == "fwd":
        return srnl.lib().srnl_linear_fwd(None, M, K, N, pp, None, None)
    return srnl.lib().srnl_linear_bwd(None, None, M, K, N, pp, None, None, None, dw, db, None, 0)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(params=False), PTR), (dict(M=-1), ARG), (dict(K=0), ARG), (dict(N=-4), ARG),
    (dict(act=3), ARG), (dict(act=-1), ARG), (dict(M=1 << 60), ARG), (dict(M=1 << 40, N=4096), ARG),
    (dict(M=1 << 31, K=1, N=1), ARG),
    (dict(types=(2, 0, 0, 0)), DTYPE), (dict(types=(0, 7, 0, 0)), DTYPE),
    (dict(types=(0, 0, 0, -1)), DTYPE), (dict(types=(0, 0, 4, 0), res=16), DTYPE), (dict(M=0), OK)])
def test_linear_errors(fn, kw, status):
    assert linear(fn, **kw) == status


def test_linear_pointer_and_workspace_errors():
    assert linear("fwd") == PTR
    assert linear("bwd") == OK                          # nothing wanted
    assert linear("bwd", db=16) == PTR                  # the bias gradient needs the weight's
    assert linear("bwd", M=100000, K=64, N=64, act=1, dw=16) == WS
    L = srnl.lib()
    p = srnl.LinearParams(None, None, None, 0, 0, 0, 0, 1, None)
    n = L.srnl_linear_bwd_workspace_bytes(9000, 512, 1024, ctypes.byref(p))
    assert n >= 4 * 9000 * 1024                         # dz
    assert L.srnl_linear_bwd_workspace_bytes(0, 64, 128, ctypes.byref(p)) == 0
    assert L.srnl_linear_bwd_workspace_bytes(5, 0, 128, ctypes.byref(p)) == 0
    assert L.srnl_linear_bwd_workspace_bytes(5, 8, 128, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), ARG), (dict(H=-1), ARG), (dict(W=-1), ARG), (dict(C=0), ARG),
    (dict(B=1 << 30, H=1 << 30, W=1 << 4), ARG), (dict(W=1 << 28, C=64), ARG), (dict(t=2), DTYPE),
    (dict(), PTR), (dict(B=0), OK), (dict(H=0), OK), (dict(W=0), OK)])
def test_dwconv_errors(kw, status):
    k = dict(B=1, H=2, W=2, C=8, t=0)
    k.update(kw)
    B, H, W, C, t = (k[n] for n in ("B", "H", "W", "C", "t"))
    L = srnl.lib()
    assert L.srnl_dwconv_fwd(None, B, H, W, C, t, None, None, None, 0, None, 0, 0, None, None) == status
    assert L.srnl_dwconv_bwd(None, t, None, B, H, W, C, 0, None, None, None, None, None, None, 0,
                             None) == status
    if status != OK and kw:
        assert L.srnl_dwconv_bwd_workspace_bytes(B, H, W, C) == 0 or "t" in kw


def test_dwconv_workspace_error():
    L = srnl.lib()
    assert L.srnl_dwconv_bwd_workspace_bytes(2, 5, 7, 12) > 0
    assert L.srnl_dwconv_bwd(None, 0, None, 2, 5, 7, 12, 0, None, None, None, 16, None, 16, 4,
                             None) == WS


def test_binding_checks_shapes_types_and_devices():
    t = torch.zeros
    x, w = t(4, 24), t(40, 24)
    g = t(24)
    for bad in (lambda: srnl.layer_norm_fwd(x, t(23), g), lambda: srnl.layer_norm_fwd(x, g, t(24).half()),
                lambda: srnl.layer_norm_fwd(x.half(), g, g),
                lambda: srnl.layer_norm_bwd(t(5, 24), x, g, t(4), t(4)),
                lambda: srnl.layer_norm_bwd(x, x, g, t(5), t(4)),
                lambda: srnl.layer_norm_bwd(x, x, g, t(4), t(4), dx_add=t(4, 23)),
                lambda: srnl.linear_fwd(t(4, 23), w), lambda: srnl.linear_fwd(x, w, t(24)),
                lambda: srnl.linear_fwd(x, w, act="relu"), lambda: srnl.linear_fwd(x, w, act=7),
                lambda: srnl.linear_fwd(x, w, residual=t(4, 24)),
                lambda: srnl.linear_bwd(t(4, 24), x, w), lambda: srnl.linear_bwd(t(4, 40), x, w, act="gelu"),
                lambda: srnl.linear_bwd(t(4, 40), x, w, t(4, 41), act="gelu"),
                lambda: srnl.linear_bwd(t(4, 40), x, w, dx_add=x.bfloat16()),
                lambda: srnl.linear_bwd(t(4, 40), x, w, need_dw=False),
                lambda: srnl.dwconv_fwd(t(1, 2, 2, 24), t(24, 9)),
                lambda: srnl.dwconv_fwd(t(1, 2, 2, 24), t(24, 3, 3), t(3)),
                lambda: srnl.dwconv_fwd(t(1, 2, 2, 24), t(24, 3, 3), g, t(1, 2, 24)),
                lambda: srnl.dwconv_bwd(t(1, 2, 3, 24), t(1, 2, 2, 24), t(24, 3, 3)),
                # CPU tensors of the right shapes: there is no CPU path
                lambda: srnl.layer_norm_fwd(x, g, g), lambda: srnl.linear_fwd(x, w),
                lambda: srnl.dwconv_fwd(t(1, 2, 2, 24), t(24, 3, 3))):
        with pytest.raises(ValueError):
            bad()
