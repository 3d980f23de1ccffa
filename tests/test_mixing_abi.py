"""Refusals of group norm, dropout and the gated delta rule, on the CPU: invalid
sizes, types and pointers return their status before any device work, and the
binding checks shapes first."""
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

from self_referential_memory_amd import srnl

ARG, DTYPE, PTR, WS, OK = (srnl.SRNL_ERR_ARG, srnl.SRNL_ERR_DTYPE, srnl.SRNL_ERR_PTR,
                           srnl.SRNL_ERR_WORKSPACE, srnl.SRNL_OK)
INF, NAN = float("inf"), float("nan")


def gnorm(fn, B=2, S=5, C=8, G=2, i=0, o=0, eps=1e-5, act=0, ws=None, nws=0):
    L = srnl.lib()
    if fn == "fwd":
        return L.srnl_group_norm_fwd(None, B, S, C, G, i, None, None, eps, act, o, None, None, None, ws, nws, None)
    return L.srnl_group_norm_bwd(None, o, None, B, S, C, G, i, None, None, None, None, act, None, None, None, None, ws,
                                 nws, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), ARG), (dict(S=-1), ARG), (dict(C=0), ARG), (dict(G=0), ARG), (dict(G=3), ARG), (dict(G=-2), ARG),
    (dict(G=16), ARG), (dict(C=1 << 21, G=1), ARG), (dict(B=1 << 20, C=16), ARG), (dict(S=1 << 41), ARG),
    (dict(B=1 << 12, C=1 << 10, S=1 << 39), ARG), (dict(act=3), ARG), (dict(act=-1), ARG), (dict(i=2), DTYPE),
    (dict(o=-1), DTYPE), (dict(B=0), OK), (dict(S=0), OK)])
def test_group_norm_errors(fn, kw, status):
    assert gnorm(fn, **kw) == status
    assert (srnl.lib().srnl_last_error().decode() == "") == (status == OK)
    if status == ARG and "act" not in kw:
        k = dict(B=2, S=5, C=8, G=2)
        k.update({n: v for n, v in kw.items() if n in k})
        assert srnl.lib().srnl_group_norm_fwd_workspace_bytes(k["B"], k["S"], k["C"], k["G"]) == 0
        assert srnl.lib().srnl_group_norm_bwd_workspace_bytes(k["B"], k["S"], k["C"], k["G"]) == 0


def test_group_norm_eps_pointers_and_workspace():
    for eps in (0.0, -1.0, NAN, INF):
        assert gnorm("fwd", eps=eps) == ARG
    assert gnorm("fwd") == PTR                              # slices: no workspace
    assert gnorm("bwd") == WS and gnorm("bwd", ws=16, nws=4 * 2 * 2 * 8) == PTR
    long = dict(B=1, S=100000, C=64, G=16)                  # slabs
    n = srnl.lib().srnl_group_norm_fwd_workspace_bytes(1, 100000, 64, 16)
    assert n > 0 and gnorm("fwd", **long) == WS and gnorm("fwd", **long, ws=16, nws=n - 1) == WS
    assert gnorm("fwd", **long, ws=16, nws=n) == PTR


def drop(fn, n=16, p=0.5, i=0, o=0, res=None, res_t=0, x=None, counter=None):
    L = srnl.lib()
    if fn == "fwd":
        return L.srnl_dropout_fwd(x, i, n, p, 1, 2, counter, res, res_t, o, None, None)
    return L.srnl_dropout_bwd(x, o, n, p, 1, 2, counter, res, i, None, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(n=1 << 60), ARG), (dict(p=1.0), ARG), (dict(p=-1e-9), ARG), (dict(p=NAN), ARG),
    (dict(p=INF), ARG), (dict(i=2), DTYPE), (dict(o=-1), DTYPE), (dict(), PTR), (dict(x=24), PTR), (dict(n=0), OK)])
def test_dropout_errors(fn, kw, status):
    assert drop(fn, **kw) == status
    assert drop("fwd", res=16, res_t=7) == DTYPE


def delta(fn="fwd", params=True, ws=None, nws=0, rec=None, nrec=0, out=None, **kw):
    L = srnl.lib()
    p = srnl.GatedDeltaParams(B=2, T=70, Hk=2, H=4, Dk=16, Dv=24, dtype=0, scale=0.25, norm_eps=0.0)
    for n, v in kw.items():
        setattr(p, n, v)
    pp = ctypes.byref(p) if params else None
    if fn == "sizes":
        return (L.srnl_gated_delta_fwd_workspace_bytes(pp), L.srnl_gated_delta_bwd_workspace_bytes(pp),
                L.srnl_gated_delta_record_bytes(pp))
    if fn == "step":
        return L.srnl_gated_delta_step(pp, out, None)
    if fn == "fwd":
        return L.srnl_gated_delta_fwd(pp, out, None, rec, nrec, ws, nws)
    return L.srnl_gated_delta_bwd(pp, None, None, rec, nrec, None, None, None, None, None, None, ws, nws)


BAD = [(dict(params=False), PTR), (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(Hk=0), ARG), (dict(H=0), ARG),
       (dict(H=3), ARG), (dict(H=-4), ARG), (dict(Dk=0), ARG), (dict(Dk=12), ARG), (dict(Dk=136), ARG),
       (dict(Dv=4), ARG), (dict(Dv=264), ARG), (dict(Dv=-8), ARG), (dict(H=1 << 21), ARG), (dict(q_stride=24), ARG),
       (dict(k_stride=33), ARG), (dict(v_stride=88), ARG), (dict(v_stride=100), ARG), (dict(q_stride=-32), ARG),
       (dict(H=1 << 18, Dk=24, Dv=8), ARG), (dict(q_stride=(1 << 22) + 8), ARG), (dict(B=1 << 30), ARG), (dict(T=(1 << 31) - 1, B=4), ARG),
       (dict(dtype=2), DTYPE), (dict(scale=NAN), ARG), (dict(scale=INF), ARG), (dict(norm_eps=-1e-9), ARG),
       (dict(norm_eps=NAN), ARG), (dict(norm_eps=INF), ARG)]


@pytest.mark.parametrize("fn", ["step", "fwd", "bwd"])
@pytest.mark.parametrize("kw,status", BAD + [(dict(B=0), OK)])
def test_gated_delta_errors(fn, kw, status):
    assert delta(fn, **kw) == status
    if status != OK:
        assert delta("sizes", **kw) == (0, 0, 0)


def test_gated_delta_workspaces_and_pointers():
    fwd, bwd, rec = delta("sizes")
    chunks = 2 * 4 * 2
    assert rec == chunks * 4 * (64 * 24 + 16 * 24) and bwd > fwd > 0
    assert delta("sizes", T=0) == (0, 0, 0) and delta("sizes", B=0) == (0, 0, 0)
    assert delta("step") == PTR
    assert delta("fwd") == WS and delta("fwd", ws=16, nws=fwd - 1) == WS and delta("fwd", ws=16, nws=fwd) == PTR
    assert delta("fwd", ws=16, nws=fwd, rec=16, nrec=rec - 1) == WS
    assert delta("bwd") == WS and delta("bwd", ws=16, nws=bwd) == WS
    assert delta("bwd", ws=16, nws=bwd, rec=16, nrec=rec - 1) == WS
    assert delta("bwd", ws=16, nws=bwd, rec=16, nrec=rec) == PTR


def test_binding_checks_shapes_types_and_devices():
    t = torch.zeros
    x, g = t(2, 5, 8), t(8)
    q, v, s = t(2, 3, 1, 16), t(2, 3, 2, 24), t(2, 2, 16, 24)
    w = t(2, 3, 2)
    n = t(2, dtype=torch.int32)

    def fwd(q=q, k=q, v=v, g=w, b=w, **kw):
        return srnl.gated_delta_fwd(q, k, v, g, b, **kw)

    for bad in (lambda: srnl.group_norm_fwd(x, 2, t(7), g), lambda: srnl.group_norm_fwd(x, 2, g, g.double()),
                lambda: srnl.group_norm_fwd(x, 2, g, g, act="relu"), lambda: srnl.group_norm_fwd(x.half(), 2, g, g),
                lambda: srnl.group_norm_fwd(g, 2, g, g),
                lambda: srnl.group_norm_bwd(t(2, 5, 7), x, 2, g, g, t(2, 2), t(2, 2)),
                lambda: srnl.group_norm_bwd(x, x, 2, g, g, t(2, 3), t(2, 2)),
                lambda: srnl.group_norm_bwd(x, x, 2, g, g, t(2, 2), t(2, 2), dx_add=x.bfloat16()),
                lambda: srnl.dropout_fwd(x, 0.5, 1, residual=g), lambda: srnl.dropout_fwd(x.half(), 0.5, 1),
                lambda: srnl.dropout_fwd(x, 0.5, 1, counter=t(1)),
                lambda: srnl.dropout_bwd(x, 0.5, 1, dx_add=x.bfloat16()),
                lambda: fwd(k=t(2, 3, 1, 24)), lambda: fwd(k=q.bfloat16()), lambda: fwd(v=t(2, 4, 2, 24)),
                lambda: fwd(g=w.double()), lambda: fwd(b=t(2, 3, 1)), lambda: fwd(state=t(2, 2, 24, 16)),
                lambda: fwd(state=s.bfloat16()), lambda: fwd(lengths=n.long()), lambda: fwd(lengths=t(3, dtype=torch.int32)),
                lambda: fwd(q=t(2, 3, 16)), lambda: fwd(v=t(2, 3, 48)),
                lambda: srnl.gated_delta_step(q, q, v, w, w, t(2, 2, 16, 16)),
                lambda: srnl.gated_delta_bwd(t(2, 3, 2, 16), q, q, v, w, w, t(4, dtype=torch.uint8)),
                lambda: srnl.gated_delta_bwd(v, q, q, v, w, w, t(4)),
                lambda: srnl.gated_delta_bwd(v, q, q, v, w, w, t(4, dtype=torch.uint8), dstate=t(2, 2, 24, 16))):
        with pytest.raises(ValueError) as e:
            bad()
        assert "GPU" not in str(e.value)
    for bad in (lambda: srnl.group_norm_fwd(x, 2, g, g), lambda: srnl.dropout_fwd(x, 0.5, 1), lambda: fwd(),
                lambda: srnl.gated_delta_step(q, q, v, w, w, s)):
        with pytest.raises(ValueError, match="GPU"):        # there is no CPU path
            bad()
    for name in ("q", "k", "v"):
        u = t(2, 3, 2, 48)[..., ::2]
        with pytest.raises(ValueError, match="contiguous"):
            srnl._token_stride(u, name)
    assert srnl._token_stride(t(2, 3, 64)[..., 16:48].unflatten(2, (2, 16)), "q") == 64
    assert srnl._token_stride(t(2, 3, 64)[:1, :, 16:48].unflatten(2, (2, 16)), "q") == 64
    assert srnl._token_stride(t(2, 1, 64)[..., 16:48].unflatten(2, (2, 16)), "q") == 64


@pytest.fixture
def calls(monkeypatch):
    """Every forward entry point returns zeros of its output's shape."""
    def norm(x, groups, gain, bias, eps=1e-5, *, act="none", out_dtype=None, stats=False, **kw):
        y = torch.zeros(x.shape)
        return (y, torch.zeros(x.shape[0], groups), torch.ones(x.shape[0], groups)) if stats else y

    def rule(q, k, v, g, beta, *, state=None, record=False, **kw):
        r = torch.zeros(v.shape), torch.zeros(v.shape[0], v.shape[2], q.shape[3], v.shape[3])
        return r + (torch.zeros(1, dtype=torch.uint8),) if record else r

    monkeypatch.setattr(srnl, "group_norm_fwd", norm)
    monkeypatch.setattr(srnl, "dropout_fwd", lambda x, *a, **kw: torch.zeros(x.shape))
    monkeypatch.setattr(srnl, "gated_delta_fwd", rule)
    x, gn = torch.randn(2, 5, 8), torch.randn(8)
    q, v, w = torch.randn(2, 3, 1, 16), torch.randn(2, 3, 2, 24), torch.randn(2, 3, 2)
    return {"group_norm": (lambda *t: srnl.group_norm(t[0], 2, *t[1:]), [x, gn, gn.clone()]),
            "dropout": (lambda *t: srnl.dropout(t[0], 0.5, 1, residual=t[1]), [x, x.clone()]),
            "gated_delta": (lambda *t: srnl.gated_delta(*t)[0],
                            [q, q.clone(), v, w, w.clone(), torch.randn(2, 2, 16, 24)])}


@pytest.mark.parametrize("op", ["group_norm", "dropout", "gated_delta"])
def test_autograd_nodes_only_where_wanted_and_no_forward_mode(calls, op):
    f, args = calls[op]
    assert f(*args).grad_fn is None
    for i in range(len(args)):
        leaf = [t.clone().requires_grad_(j == i) for j, t in enumerate(args)]
        assert f(*leaf).grad_fn is not None
        with torch.no_grad():
            assert f(*leaf).grad_fn is None
        with forward_ad.dual_level():
            dual = list(args)
            dual[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(RuntimeError, match="jvp"):
                f(*dual)
