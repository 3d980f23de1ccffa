"""The gated delta rule against the rule token by token in float64.

Bounds, fixed before the first run. u = 2^-24, r(t) half a step of the output's
type (bf16 2^-8, fp32 2^-24). With beta |k|^2 <= 2 and g <= 0 a token's
transition does not lengthen a vector, so errors made at earlier tokens do not
grow. A token makes products of Dk terms, its update and its readout: in norm
each is off by at most (Dk + 8) u of the state's norm, twice that if sums
truncate; T tokens by 4 T (Dk + 8) u. Norms are taken per item and head. The
scale is the larger of the reference's norm and its mean over the heads; for
outputs it is the norm of the terms scale |S| |q| that they are sums of: a sum's
roundings are relative to its terms, and the one token of a single head may
leave next to nothing of them (q.k = 0).

In chunks of 64 the rule is five chained products: rows of at most Dk, 64 and 64
terms, through an inverse that stretches by at most a few (4 is allowed for). fp32
is off by 4 x 4 (Dk + 136) u a chunk; with bf16 inputs each operand between is
right to 2^-17, a product of two to 2^-16 of the norms, 4 x 4 x 2^-16 a chunk
besides. The backward pass makes as many products again, of values that carry the
forward's error, and adds its own: three times that.
"""
import pytest
import torch

from self_referential_memory_amd import srnl
from tests import delta_oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def say(*a):
    print("[delta]", *a, flush=True)


def on_gpu(d):
    return {n: None if t is None else t.to(DEV) for n, t in d.items()}


def close(got, ref, tol, what, heads, terms=None):
    """Per item and head (axis `heads` of ref): |got - ref| <= tol times the
    scale plus half a step of the reference's norm."""
    g, r = got.detach().cpu().double(), ref
    assert g.shape == r.shape, what
    dims = [i for i in range(r.dim()) if i not in (0, heads)]
    err = (g - r).square().sum(dims).sqrt()
    norm = r.square().sum(dims).sqrt()
    size = torch.maximum(norm, norm.mean()) if terms is None else terms.square().sum(dims).sqrt()
    over = err - tol * size - HALF[got.dtype] * norm - 1e-30
    assert bool((over <= 0).all()), f"{what}: off by {(err / (size + 1e-30)).max().item():.3e}, bound {tol:.3e}"


def step_tol(T, Dk):
    return 4 * T * (Dk + 8) * U


STEP = [  # B, T, Hk, H, Dk, Dv, norm, lengths
    (1, 1, 1, 1, 8, 8, True, None), (3, 1, 2, 4, 128, 128, True, None), (2, 5, 1, 3, 64, 72, True, (5, 2)),
    (4, 3, 2, 2, 40, 200, False, (0, 1, 3, 9)), (2, 2, 1, 2, 120, 256, True, (-4, 2)), (2, 7, 3, 3, 16, 64, False, None),
    (1, 4, 1, 1, 104, 8, True, None),
    # enough heads for the wider blocks
    (64, 2, 2, 4, 128, 72, True, None), (64, 1, 4, 4, 32, 64, False, None), (64, 3, 4, 4, 64, 40, True, None)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("case", STEP, ids=str)
def test_step(case, dtype, state):
    B, T, Hk, H, Dk, Dv, norm, lengths = case
    say("step", case, dtype, state)
    d = delta_oracle.inputs(7, B, T, Hk, H, Dk, Dv, dtype, norm=norm, state=state, lengths=lengths)
    eps = 1e-6 if norm else 0.0
    ref, S, terms = delta_oracle.reference(d, norm_eps=eps)
    x = on_gpu(d)
    st = x["state"] if state else torch.zeros(B, H, Dk, Dv, device=DEV)
    before, new = st.clone(), torch.empty_like(st)
    out, S1 = srnl.gated_delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], st, lengths=x["lengths"],
                                    norm_eps=eps, state_out=new)
    assert S1 is new and torch.equal(st, before)
    close(out, ref, step_tol(T, Dk), "out", 2, terms)
    close(S1, S, step_tol(T, Dk), "state", 1)
    # in place, the same bits
    out2, S2 = srnl.gated_delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], st, lengths=x["lengths"],
                                     norm_eps=eps)
    assert S2 is st and torch.equal(S2, new) and torch.equal(out2, out)
    if lengths is not None:
        for b, n in enumerate(lengths):
            assert not out[b, max(n, 0):].any()
            if n <= 0:
                assert torch.equal(S1[b], before[b])


def chunk_tol(T, Dk, dtype):
    chunks = max(1, -(-T // 64))
    return 16 * chunks * ((Dk + 136) * U + (2.0 ** -16 if dtype == BF16 else 0.0))


CHUNKED = [  # B, T, Hk, H, Dk, Dv, norm, lengths
    (1, 1, 1, 1, 8, 8, True, None), (2, 2, 1, 2, 32, 32, True, None), (1, 63, 2, 2, 64, 64, False, None),
    (2, 64, 1, 3, 128, 128, True, None), (1, 65, 2, 4, 40, 72, True, None), (2, 200, 2, 2, 24, 200, True, (200, 131)),
    (5, 130, 1, 2, 96, 48, False, (0, 1, 64, 65, 130)), (1, 257, 3, 6, 128, 256, True, None),
    (3, 90, 1, 1, 16, 8, True, (500, -3, 89)), (2, 129, 2, 2, 56, 40, False, None),
    # enough heads for slabs of 32 columns
    (64, 70, 2, 4, 32, 32, True, None), (65, 65, 4, 4, 64, 40, False, None), (33, 66, 4, 8, 128, 48, True, None)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("case", CHUNKED, ids=str)
def test_forward_and_backward(case, dtype, state):
    B, T, Hk, H, Dk, Dv, norm, lengths = case
    say("chunks", case, dtype, state)
    d = delta_oracle.inputs(11, B, T, Hk, H, Dk, Dv, dtype, norm=norm, state=state, lengths=lengths)
    gen = torch.Generator().manual_seed(3)
    dout = torch.randn((B, T, H, Dv), generator=gen).to(dtype)
    dstate = 0.3 * torch.randn((B, H, Dk, Dv), generator=gen) if state else None
    eps = 1e-6 if norm else 0.0
    ref, S, terms, grads = delta_oracle.reference(d, norm_eps=eps, dout=dout, dstate=dstate)
    x = on_gpu(d)
    kw = dict(state=x["state"], lengths=x["lengths"], norm_eps=eps)
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    out, S1, rec = srnl.gated_delta_fwd(*args, record=True, **kw)
    tol = chunk_tol(T, Dk, dtype)
    close(out, ref, tol, "out", 2, terms)
    close(S1, S, tol, "state", 1)
    out2, S2 = srnl.gated_delta_fwd(*args, **kw)          # without a record, the same bits
    assert torch.equal(out, out2) and torch.equal(S1, S2)
    got = srnl.gated_delta_bwd(dout.to(DEV), *args, rec, dstate=None if dstate is None else dstate.to(DEV), **kw)
    for name, t in zip(("q", "k", "v", "g", "beta", "state"), got):
        if t is None:
            assert not state and name == "state"
            continue
        close(t, grads[name], 3 * tol, "d" + name, 1 if name == "state" else 2)
    if lengths is not None:
        for b, n in enumerate(lengths):
            n = min(max(n, 0), T)
            assert not any(t[b, n:].any() for t in (out, *got[:5]))
            if n == 0 and state:
                assert torch.equal(S1[b], x["state"][b]) and torch.equal(got[5][b], dstate[b].to(DEV))
    again = srnl.gated_delta_bwd(dout.to(DEV), *args, rec, dstate=None if dstate is None else dstate.to(DEV), **kw)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
