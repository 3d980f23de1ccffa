"""A residual branch that mixes a map's tokens, from the operators as a model
would use them: group norm with SiLU, one projection to q, k, v and the gates,
the gated delta rule, the output projection, dropout into the residual.

The reference is the same branch in float64. Errors in norm, relative: each
linear layer and norm sums at most 512 terms in fp32 (2 x 520 u = 6e-5, u =
2^-24) and the rule is off by its own bound (its tests: 16 (Dk + 136) u a chunk
of 64, 2e-4 for one chunk at Dk = 16); with fp32 tensors the five steps forward
stay below 1e-3 of their inputs' size, the gradients, as long again and through
both, below 5e-3.
"""
import pytest
import torch

from self_referential_memory_amd import srnl
from tests import delta_oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HK, H, DK, DV, C, G = 1, 2, 16, 24, 48, 6
P, SEED = 0.25, 77
PAD = 4                                    # rows of the projection are whole pieces of 8
WIDTH = 2 * HK * DK + H * DV + 2 * H + PAD


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    return {"gain": 1 + 0.2 * r(C), "bias": 0.2 * r(C), "w_in": r(WIDTH, C) / C ** 0.5, "b_in": 0.1 * r(WIDTH),
            "w_out": r(C, H * DV) / (H * DV) ** 0.5}


def cut(z):
    """q, k, v and the gates of a projection [B, T, WIDTH]."""
    q, k, v, g, b, _ = z.split((HK * DK, HK * DK, H * DV, H, H, PAD), -1)
    return q.unflatten(2, (HK, DK)), k.unflatten(2, (HK, DK)), v.unflatten(2, (H, DV)), g, b


def branch(x, w, state=None, lengths=None, offset=0):
    n = srnl.group_norm(x, G, w["gain"], w["bias"], act="silu")
    z = srnl.linear(n, w["w_in"], w["b_in"])
    q, k, v, g, b = cut(z)
    g = -torch.nn.functional.softplus(g).contiguous()
    y, S = srnl.gated_delta(q, k, v, g, b.sigmoid().contiguous(), state, lengths=lengths, norm_eps=1e-6)
    o = srnl.linear(y.flatten(2), w["w_out"])
    return srnl.dropout(o, P, SEED, offset, residual=x), S


def reference(x, w, keep, state=None, lengths=None):
    B, T, _ = x.shape
    X = x.reshape(B, T, G, C // G)
    m = X.mean((1, 3), keepdim=True)
    r = (X - m).square().mean((1, 3), keepdim=True).add(1e-5).rsqrt()
    n = ((X - m) * r).reshape(B, T, C) * w["gain"] + w["bias"]
    n = n * n.sigmoid()
    q, k, v, g, b = cut(n @ w["w_in"].t() + w["b_in"])
    y, S, _ = delta_oracle.rule(q, k, v, -torch.nn.functional.softplus(g), b.sigmoid(), state, lengths, None, 1e-6)
    return x + torch.where(keep, (y.flatten(2) @ w["w_out"].t()) / (1 - P), 0.0), S


def off(got, ref):
    return ((got.detach().cpu().double() - ref).norm() / ref.norm()).item()


def test_training_step():
    B, T = 2, 100
    x = torch.randn(B, T, C, generator=torch.Generator().manual_seed(1))
    wt = torch.randn(B, T, C, generator=torch.Generator().manual_seed(2))
    w = weights()
    lengths = torch.tensor([100, 61], dtype=torch.int32)
    dev = {n: t.to(DEV).requires_grad_() for n, t in w.items()}
    xd = x.to(DEV).requires_grad_()
    y, S = branch(xd, dev, lengths=lengths.to(DEV))
    ones = torch.ones(B, T, C, device=DEV)
    keep = srnl.dropout_fwd(ones, P, SEED) > 0
    w64 = {n: t.double().requires_grad_() for n, t in w.items()}
    x64 = x.double().requires_grad_()
    ry, rS = reference(x64, w64, keep.cpu(), lengths=lengths)
    assert off(y, ry.detach()) < 1e-3 and off(S, rS.detach()) < 1e-3
    names = list(w)
    got = torch.autograd.grad((y * wt.to(DEV)).sum(), [xd] + [dev[n] for n in names])
    ref = torch.autograd.grad((ry * wt.double()).sum(), [x64] + [w64[n] for n in names])
    for n, a, b in zip(["x"] + names, got, ref):
        assert off(a, b) < 5e-3, n


def test_prompt_then_tokens():
    """A prompt through the rule, then its next tokens one by one: the same
    outputs as the whole sequence at once."""
    B, T, more = 3, 70, 5
    g = torch.Generator().manual_seed(3)
    z = torch.randn(B, T + more, WIDTH, generator=g).to(DEV).bfloat16()
    q, k, v, gate, b = cut(z)
    gate, b = -torch.nn.functional.softplus(gate.float()).contiguous(), b.float().sigmoid().contiguous()
    whole, last = srnl.gated_delta_fwd(q, k, v, gate, b, norm_eps=1e-6)
    head = z[:, :T].contiguous()
    q1, k1, v1, _, _ = cut(head)
    out, state = srnl.gated_delta_fwd(q1, k1, v1, gate[:, :T].contiguous(), b[:, :T].contiguous(), norm_eps=1e-6)
    outs = [out]
    for t in range(T, T + more):
        q1, k1, v1, _, _ = cut(z[:, t:t + 1].contiguous())
        o, state = srnl.gated_delta_step(q1, k1, v1, gate[:, t:t + 1].contiguous(), b[:, t:t + 1].contiguous(), state,
                                         norm_eps=1e-6)
        outs.append(o)
    joined = torch.cat(outs, 1)
    # bf16 outputs of values that agree to 1e-5: at most one step (2^-7) apart
    assert bool(((joined.float() - whole.float()).abs() <= 2.0 ** -7 * whole.float().abs() + 1e-5).all())
    assert off(state, last.cpu().double()) < 1e-4
