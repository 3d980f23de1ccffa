"""How far a NaN or an infinity reaches in the gated delta rule over whole
sequences: what lies outside has the bits that it has without it. The step takes
it where the formulas do."""
import pytest
import torch

from self_referential_memory_amd import srnl
from tests import delta_oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
B, T, HK, H, DK, DV = 3, 300, 2, 4, 40, 48
ITEM, HEAD, COL = 1, 2, 5             # where the bad value is: head 2 takes q and k of head 1
TOKENS = (64 + 20, 64 + 50, 128)      # in either half of a chunk, and a chunk's first


def inputs(dtype):
    d = delta_oracle.inputs(80, B, T, HK, H, DK, DV, dtype, state=True)
    gen = torch.Generator().manual_seed(81)
    d["dout"] = torch.randn((B, T, H, DV), generator=gen).to(dtype)
    d["dstate"] = torch.randn((B, H, DK, DV), generator=gen)
    return {n: None if t is None else t.to(DEV) for n, t in d.items()}


def both(x):
    args = tuple(x[n] for n in ("q", "k", "v", "g", "beta"))
    out, S, rec = srnl.gated_delta_fwd(*args, state=x["state"], norm_eps=1e-6, record=True)
    g = srnl.gated_delta_bwd(x["dout"], *args, rec, state=x["state"], dstate=x["dstate"], norm_eps=1e-6)
    return dict(zip(("out", "S", "dq", "dk", "dv", "dg", "dbeta", "dstate"), (out, S, *g)))


def same(a, b):
    """Bits: NaNs of both count as equal."""
    return torch.equal(a.nan_to_num(nan=7.25), b.nan_to_num(nan=7.25))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta", "state", "dout"])
def test_reach(where, dtype, bad):
    x = inputs(dtype)
    clean = both(x)
    assert all(t.isfinite().all() for t in clean.values())
    for tok in TOKENS if where != "state" else (0,):
        print("[delta nonfinite]", where, dtype, bad, tok, flush=True)
        y = {n: None if t is None else t.clone() for n, t in x.items()}
        heads = [HEAD]
        if where in ("q", "k"):
            y[where][ITEM, tok, 1, 3] = bad
            heads = [2, 3]
        elif where in ("v", "dout"):
            y[where][ITEM, tok, HEAD, COL] = bad
        elif where == "state":
            y[where][ITEM, HEAD, 3, COL] = bad
        else:
            y[where][ITEM, tok, HEAD] = bad
        got = both(y)
        start, end = tok // 64 * 64, tok // 64 * 64 + 64
        others = [h for h in range(H) if h not in heads]
        items = [b for b in range(B) if b != ITEM]
        for n, t in got.items():
            c = clean[n]
            per_item = 1 if n in ("S", "dstate") else 2            # axis of heads
            assert same(t[items], c[items]), n                     # other items
            rest = [0] if n in ("dq", "dk") else others            # other heads (of q and k)
            index = torch.tensor(rest, device=DEV)
            assert same(t[ITEM].index_select(per_item - 1, index), c[ITEM].index_select(per_item - 1, index)), n
        out, want = got["out"][ITEM], clean["out"][ITEM]
        assert same(out[:start], want[:start])
        cols = [j for j in range(DV) if j != COL]
        if where in ("v", "state"):
            assert same(out[..., cols], want[..., cols])
            assert same(got["S"][ITEM][..., cols], clean["S"][ITEM][..., cols])
        if where == "q":
            keep = [t for t in range(T) if t != tok]
            assert same(out[keep], want[keep]) and same(got["S"], clean["S"])
        if where == "dout":
            assert same(got["out"], clean["out"]) and same(got["S"], clean["S"])
        if where != "dout":                                        # and there it is
            assert not out[tok, heads].isfinite().all()
        grads = ("dq", "dk", "dv", "dg", "dbeta")
        if where == "v":
            assert all(same(got[n][ITEM, :start], clean[n][ITEM, :start]) for n in grads)
        if where in ("q", "dout"):
            assert all(same(got[n][ITEM, end:], clean[n][ITEM, end:]) for n in grads)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_step_keeps_earlier_tokens(dtype):
    x = inputs(dtype)
    args = [x[n][:, :6].contiguous() for n in ("q", "k", "v", "g", "beta")]
    want, S = srnl.gated_delta_step(*args, x["state"].clone(), norm_eps=1e-6)
    args[2][ITEM, 3, HEAD, COL] = float("nan")
    out, S1 = srnl.gated_delta_step(*args, x["state"].clone(), norm_eps=1e-6)
    assert same(out[:, :3], want[:, :3]) and out[ITEM, 3:, HEAD, COL].isnan().all()
    cols = [j for j in range(DV) if j != COL]
    assert same(out[..., cols], want[..., cols]) and same(S1[..., cols], S[..., cols])
    # a gate of -infinity starts a finite state anew, and only such a one
    args[3][ITEM, 4, HEAD] = float("-inf")
    out, _ = srnl.gated_delta_step(*args, x["state"].clone(), norm_eps=1e-6)
    assert out[ITEM, 4:, HEAD, COL].isnan().all() and out[ITEM, 4:, HEAD][..., cols].isfinite().all()
