"""The gated delta rule token by token in float64 (torch autograd gives its
gradients), and inputs for its tests."""
import torch


def rule(q, k, v, g, beta, state=None, lengths=None, scale=None, norm_eps=0.0):
    """float64 tensors in the layout of srnl.gated_delta_*: (out, last state,
    the magnitudes of the terms whose sums out is)."""
    B, T, Hk, Dk = q.shape
    H, Dv = v.shape[2:]
    scale = Dk ** -0.5 if scale is None else scale
    if norm_eps > 0:
        q, k = (t / (t.square().sum(-1, keepdim=True) + norm_eps).sqrt() for t in (q, k))
    q, k = (t.repeat_interleave(H // Hk, 2) for t in (q, k))
    S = torch.zeros(B, H, Dk, Dv, dtype=torch.float64) if state is None else state
    n = torch.full((B,), T) if lengths is None else lengths.clamp(0, T)
    out, terms = [], []
    for t in range(T):
        live = (t < n)[:, None, None]
        A = S * g[:, t].exp()[..., None, None]
        e = v[:, t] - torch.einsum("bhkv,bhk->bhv", A, k[:, t])
        N = A + torch.einsum("bhk,bhv->bhkv", k[:, t], beta[:, t, :, None] * e)
        o = scale * torch.einsum("bhkv,bhk->bhv", N, q[:, t])
        # chosen, not multiplied: what lies past the end may be anything
        S = torch.where(live[..., None], N, S)
        out.append(torch.where(live, o, torch.zeros_like(o)))
        a = abs(scale) * torch.einsum("bhkv,bhk->bhv", N.detach().abs(), q[:, t].detach().abs())
        terms.append(torch.where(live, a, torch.zeros_like(a)))
    if not T:
        return v.new_zeros(v.shape), S, v.new_zeros(v.shape)
    return torch.stack(out, 1), S, torch.stack(terms, 1)


def inputs(seed, B, T, Hk, H, Dk, Dv, dtype, *, norm=True, state=False, lengths=None, decay=1.0):
    """CPU tensors: q, k, v in dtype, g, beta, the state in fp32."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    unit = 1.0 if norm else Dk ** -0.5
    d = {"q": (normal(B, T, Hk, Dk) * unit).to(dtype), "k": (normal(B, T, Hk, Dk) * unit).to(dtype),
         "v": normal(B, T, H, Dv).to(dtype),
         "g": -decay * torch.rand((B, T, H), generator=gen).square(),
         "beta": torch.sigmoid(normal(B, T, H)),
         "state": 0.3 * normal(B, H, Dk, Dv) if state else None,
         "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32)}
    return d


def reference(d, scale=None, norm_eps=0.0, dout=None, dstate=None):
    """out, last state and out's terms in float64; with dout also the gradients,
    by name."""
    names = [n for n in ("q", "k", "v", "g", "beta", "state") if d[n] is not None]
    x = {n: d[n].double().requires_grad_(dout is not None) for n in names}
    out, S, terms = rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x.get("state"), d["lengths"], scale, norm_eps)
    if dout is None:
        return out, S, terms
    loss = (out * dout.double()).sum()
    if dstate is not None:
        loss = loss + (S * dstate.double()).sum()
    grads = torch.autograd.grad(loss, [x[n] for n in names], allow_unused=True)
    return out.detach(), S.detach(), terms, {n: torch.zeros_like(x[n]) if t is None else t for n, t in zip(names, grads)}
