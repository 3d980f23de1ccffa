"""The gated delta rule in chunks of 64 tokens, in float64 but for what the
kernels hold between their products of bf16 inputs, which is cut to a sum of
bf16 words here as there: what a kernel that kept fewer words would give.

A word takes 8 bits, the sign of what is left a ninth: one word is right to
2^-9 of a value, two to 2^-18, three to 2^-27.
"""
import torch


def cut(x, words):
    """x as a sum of that many bf16 words (None: as it is)."""
    if words is None:
        return x
    left, s = x.float(), torch.zeros_like(x)
    for _ in range(words):
        w = left.bfloat16().float()
        left, s = left - w, s + w.double()
    return s


def chunked(d, scale, norm_eps, dout, dstate=None, state_words=3, out_words=3):
    """(out, last state, gradients by name) of inputs as delta_oracle's, without
    lengths. state_words: of what states and fp32 gradients depend on, out_words: of
    what only bf16 outputs do (U, P and the state as the outputs read them, and the
    matrices that multiply q and k in their gradients)."""
    def of(x):
        return cut(x, state_words)

    def of_out(x):
        return cut(x, out_words)

    B, T, Hk, Dk = d["q"].shape
    H, Dv = d["v"].shape[2:]
    N, per = -(-T // 64), H // Hk

    def chunks(t):                               # [B,T,h,...] -> [B,h,N,64,...]
        t = torch.cat((t.double(), t.new_zeros((B, 64 * N - T) + t.shape[2:]).double()), 1)
        return t.unflatten(1, (N, 64)).movedim(3, 1)

    def tokens(t):
        return t.movedim(1, 3).flatten(1, 2)[:, :T]

    qi, ki = (chunks(d[n]).repeat_interleave(per, 1) for n in ("q", "k"))
    live = chunks(torch.ones(B, T, 1))[..., None]
    if norm_eps > 0:
        rq, rk = (live / (t.square().sum(-1, keepdim=True) + norm_eps).sqrt() for t in (qi, ki))
    else:
        rq = rk = live
    v, beta, do = chunks(d["v"]), chunks(d["beta"])[..., None], chunks(dout)
    G = chunks(d["g"])[..., None].cumsum(-2)
    gam, end = G.exp(), (G[..., -1:, :] - G).exp()
    low = torch.ones(64, 64, dtype=torch.bool).tril()
    strict = low.tril(-1)
    dec = torch.where(low, (G - G.mT).exp(), 0.0)
    M = torch.where(strict, (rk * ki) @ (rk * ki).mT * dec, 0.0)
    P = scale * ((rq * qi) @ (rk * ki).mT) * dec
    X = torch.linalg.inv(torch.eye(64, dtype=torch.float64) + M * beta.mT)
    last = gam[..., -1:, :]
    S = torch.zeros(B, H, Dk, Dv, dtype=torch.float64) if d["state"] is None else d["state"].double()
    S0, E, out = [], [], []
    for c in range(N):
        kc, qc = ki[:, :, c], qi[:, :, c]
        S0.append(S)
        e = of(X[:, :, c]) @ of(v[:, :, c] - (gam * rk)[:, :, c] * (kc @ of(S)))
        out.append((scale * gam * rq)[:, :, c] * (qc @ of_out(S)) + of_out(P[:, :, c]) @ of_out(beta[:, :, c] * e))
        E.append(e)
        S = last[:, :, c] * S + kc.mT @ of((end * beta * rk)[:, :, c] * e)
    end_state = S
    D = torch.zeros_like(S) if dstate is None else dstate.double()
    D1, dV = [None] * N, [None] * N
    for c in reversed(range(N)):
        kc, qc, oc = ki[:, :, c], qi[:, :, c], do[:, :, c]
        D1[c] = D
        w = (end * beta * rk)[:, :, c] * (kc @ of(D)) + beta[:, :, c] * (of(P[:, :, c].mT) @ oc)
        dV[c] = of(X[:, :, c].mT) @ of(w)
        D = (last[:, :, c] * D + qc.mT @ of((scale * gam * rq)[:, :, c] * oc)
             + kc.mT @ of(-(gam * rk)[:, :, c] * dV[c]))
    S0, E, D1, dV = (torch.stack(t, 2) for t in (S0, E, D1, dV))
    A, Y = do @ of(E).mT, of(dV) @ of(E).mT
    oS, vS, eD = do @ of(S0).mT, of(dV) @ of(S0).mT, of(E) @ of(D1).mT
    a = torch.where(low, scale * dec * A, 0.0)
    y = torch.where(strict, dec * Y, 0.0)
    F = a * ((rq * qi) @ (rk * ki).mT) - y * ((rk * ki) @ (rk * ki).mT)
    x, r, w = scale * gam * oS, -gam * vS, end * eD
    z = -y * beta.mT
    dqh = x + of_out(a * beta.mT * rk.mT) @ ki
    dkh = beta * w + r + of_out((a * beta.mT * rq).mT) @ qi + of_out(z * rk.mT + (z * rk).mT) @ ki
    kw = (rk * ki * w).sum(-1, keepdim=True)
    dbeta = kw + F.sum(-2)[..., None]
    Fb = torch.where(strict, F * beta.mT, 0.0)
    after = Fb.sum(-1, keepdim=True) - Fb.sum(-2)[..., None] + (rq * qi * x + rk * ki * r).sum(-1, keepdim=True)
    kw = beta * kw
    dg = after.flip(-2).cumsum(-2).flip(-2) + kw.cumsum(-2) - kw + last * (of(S0) * of(D1)).sum((-1, -2))[..., None, None]
    grads = {"v": tokens(dV), "g": tokens(dg)[..., 0], "beta": tokens(dbeta)[..., 0], "state": D}
    for n, i, r, t in (("q", qi, rq, dqh), ("k", ki, rk, dkh)):
        if norm_eps > 0:
            t = t - r * i * (r * i * t).sum(-1, keepdim=True)
        grads[n] = tokens(r * t).unflatten(2, (Hk, per)).sum(3)
    return tokens(torch.stack(out, 2)), end_state, grads


# Bounds, in norm, u = 2^-24. A product's result is a sum in fp32, of at most 14
# instructions' results (K = 128: four times three pairs of words, and their join),
# each rounded by u / sqrt(3) in the mean of a partial sum that grows with the square
# root: 1.5 u; as much for the 32 products that an instruction adds: 2 u. A chunk's
# outputs and state pass three such products and as many factors and differences of
# one rounding each, sqrt(3 x 4 + 3) = 4 u; what earlier chunks left fades as the state
# itself does (e^-2 and less over a chunk here). The gradients carry that and add as
# much again, 6 u. Bounds are three times these means: 12 u and 18 u. Two words instead
# of three, each operand right to 2^-18 / sqrt(3), give 35 u and more.
U = 2.0 ** -24
TOL = {"out": 12 * U, "q": 18 * U, "k": 18 * U, "v": 18 * U}

CASES = [  # B, T, Hk, H, Dk, Dv, norm
    (2, 257, 1, 2, 128, 128, True), (2, 200, 2, 2, 24, 40, True), (3, 300, 2, 4, 64, 64, True),
    (1, 500, 1, 2, 128, 32, True), (2, 130, 1, 2, 128, 64, False), (64, 70, 2, 4, 32, 32, True)]


def case_inputs(case, dtype):
    """(inputs, dout, dstate, norm_eps, (out, last state, gradients) in float64)."""
    from tests import delta_oracle
    B, T, Hk, H, Dk, Dv, norm = case
    d = delta_oracle.inputs(61, B, T, Hk, H, Dk, Dv, dtype, norm=norm, state=True)
    gen = torch.Generator().manual_seed(62)
    dout = torch.randn((B, T, H, Dv), generator=gen).to(dtype)
    dstate = 0.3 * torch.randn((B, H, Dk, Dv), generator=gen)
    eps = 1e-6 if norm else 0.0
    out, S, _, grads = delta_oracle.reference(d, norm_eps=eps, dout=dout, dstate=dstate)
    return d, dout, dstate, eps, (out, S, grads)


def on_other_sides(got, ref, tol):
    """How many of got, bf16, are not what ref rounds to, and the most that may be:
    a value off by e before it is rounded lands on the other side of a border with
    probability |e| / step (where the border lies is any number's chance), |e| in the
    mean 0.8 of its root mean square (as normal numbers), which is tol of the token's
    and head's; and four times the deviation of a count."""
    ref = ref.detach()
    count = int((got.cpu() != ref.bfloat16()).sum())
    e = 0.8 * tol * ref.square().mean(3, keepdim=True).sqrt()
    step = 2.0 ** -7 * torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=1e-30))))
    mean = (e / step).clamp(max=1.0).sum().item()
    return count, mean + 4 * mean ** 0.5 + 1


# fp32 results, in norm over an item's and head's values, by the same counting. With
# fp32 inputs a product of K = 128 is a sum of 32 instructions' results of 4 products:
# 3.5 u in the mean; a chunk 6 u, gradients with what they carry 9 u. Four times these.
FINE = {torch.bfloat16: {"out": 16 * U, "grad": 24 * U}, torch.float32: {"out": 24 * U, "grad": 36 * U}}


def off(got, ref, heads):
    """|got - ref| in norm per item and head (axis `heads`), relative to the larger of
    the reference's norm there and its mean over them: the largest."""
    ref = ref.detach()
    dims = [i for i in range(ref.dim()) if i not in (0, heads)]
    err, norm = ((t.square().sum(dims)).sqrt() for t in (got.detach().cpu().double() - ref, ref))
    return (err / torch.maximum(norm, norm.mean())).max().item()
