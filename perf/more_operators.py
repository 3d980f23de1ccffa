"""A residual branch that mixes tokens with the gated delta rule, as calls on
the GPU: the gated delta rule over whole sequences and for single tokens,
group norm with an activation over a channels-last map in front of it, and
dropout into the residual behind it; each in inference and in training.

Sizes are those of the hierarchical backbone's maps (64 items of 56x56x64 in 2
heads of 32, ... 7x7x512), of the 1-D operator's sequences, and generic: heads
of 128, long prompts, batches of single tokens, odd and ragged sizes.

A case is one pass: "fwd" (one forward call), "train" (a forward that keeps
what the backward needs, then the backward) or "step" (tokens appended to
sequences whose states are in hand). ``run`` computes it either with elementary
torch operations in 32 bits, rounded once at the end, or (``own``) with the
package's entry points.

The operators.
  Gated delta rule, per item and head, S a Dk x Dv matrix:
    S <- exp(g_t) S;  u = beta_t (v_t - S^T k_t);  S <- S + k_t u^T;  o_t = scale S^T q_t
    with q, k divided by sqrt(|.|^2 + norm_eps) first where norm_eps > 0. Head h
    of v takes head h // (H / Hk) of q and k. Tokens at or past an item's length
    change nothing; their outputs and gradients are zero.
  Group norm: y = act(n gain + bias), n = (x - mean) rstd over a group's
    channels and all the cells of an item.
  Dropout: y = residual + x / (1 - p) where kept. Element n takes 16 bits of
    block n // 8 of Philox4x32-10 (counter: block, offset; key: seed), low half
    of word 0 first; it is dropped where they are below round(65536 p), and p is
    that multiple of 2^-16.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GN_EPS = 1e-5
QK_EPS = 1e-6
CHUNK = 64
SQRT_HALF = math.sqrt(0.5)
INV_SQRT_2PI = 1.0 / math.sqrt(2.0 * math.pi)


# ------------------------------------------------------------------- cases

def _delta(name, do, B, T, Hk, H, Dk, Dv, x, norm=True, state=False, ragged=False):
    """state: sequences start from a given state, and the last one's gradient
    is given; ragged: items have lengths of their own."""
    return {"name": name, "op": "gated_delta", "pass": do, "B": B, "T": T, "Hk": Hk, "H": H,
            "Dk": Dk, "Dv": Dv, "x": x, "norm": norm, "state": state, "ragged": ragged}


def _gn(name, do, B, S, C, G, x, out, act):
    return {"name": name, "op": "group_norm", "pass": do, "B": B, "S": S, "C": C, "G": G, "x": x,
            "out": out, "act": act}


def _drop(name, do, rows, C, x, out, p, res):
    return {"name": name, "op": "dropout", "pass": do, "rows": rows, "C": C, "x": x, "out": out,
            "p": p, "res": res}


def listed():
    return [
        # one sequence's next token, 16 heads of 128
        _delta("delta_token", "step", 1, 1, 16, 16, 128, 128, "bf16", state=True),
        # the next token of 256 sequences served together
        _delta("delta_token_batch", "step", 256, 1, 8, 16, 128, 128, "bf16", state=True),
        # the stage-1 map's cells as sequences, inference
        _delta("delta_map", "fwd", 64, 3136, 2, 2, 32, 32, "bf16"),
        # one long prompt, its last state kept
        _delta("delta_prompt", "fwd", 1, 16384, 8, 16, 128, 128, "bf16"),
        # a training step over sequences of 4096
        _delta("delta_train", "train", 4, 4096, 8, 8, 128, 128, "bf16"),
        # a ragged batch with odd heads in fp32, continued from given states
        _delta("delta_odd_train", "train", 3, 1001, 2, 6, 40, 72, "f32", norm=False, state=True,
               ragged=True),
        # one image's last-stage map
        _gn("gnorm_image", "fwd", 1, 49, 512, 32, "bf16", "bf16", "silu"),
        # the stage-1 map in training
        _gn("gnorm_stage1_train", "train", 64, 3136, 64, 16, "bf16", "bf16", "silu"),
        # a generic odd map in fp32
        _gn("gnorm_odd_train", "train", 5, 1551, 210, 7, "f32", "f32", "gelu"),
        # one image's last-stage map into its residual
        _drop("drop_image", "fwd", 49, 512, "bf16", "bf16", 0.1, "bf16"),
        # the stage-1 branch's output into the residual in training
        _drop("drop_stage1_train", "train", 200704, 64, "bf16", "bf16", 0.1, "bf16"),
        # an odd fp32 array, with no residual
        _drop("drop_odd_train", "train", 12001, 777, "f32", "bf16", 0.37, ""),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["gated_delta", "gated_delta", "group_norm", "dropout"])
    x, out = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    if op == "gated_delta":
        do = rng.choice(["step", "fwd", "train", "train"])
        Dk, Dv = 8 * _log(rng, 2, 16), 8 * _log(rng, 2, 16)
        Hk = _log(rng, 1, 8)
        H = Hk * rng.choice([1, 1, 2, 3])
        # tokens that cost no more than the listed training step, in flops and in bytes
        room = min(4 * 4096 * 8 * 128 * 128 // (H * max(Dk, Dv) * max(Dk, Dv, 64)),
                   4 * 4096 * 8 * 1408 // (6 * Hk * Dk + 5 * H * Dv) // TYPES[x].itemsize)
        if do == "step":
            B, T = _log(rng, 1, 256), rng.choice([1, 1, 2, 5])
            B = max(1, min(B, 256 * 16 * 128 * 128 // (H * Dk * Dv)))
        else:
            T = _log(rng, 1, 8192)
            B = max(1, min(_log(rng, 1, 64), room // T))
            T = max(1, min(T, room // B))
        state = do == "step" or rng.random() < 0.5
        return _unnamed(_delta("", do, B, T, Hk, H, Dk, Dv, x, norm=rng.random() < 0.7,
                               state=state, ragged=rng.random() < 0.4))
    do = rng.choice(["fwd", "train"])
    if op == "group_norm":
        G = _log(rng, 1, 32)
        C = G * _log(rng, 1, max(1, 512 // G))
        B = _log(rng, 1, 64)
        S = max(1, min(_log(rng, 1, 3136), 12_000_000 // (B * C)))
        return _unnamed(_gn("", do, B, S, C, G, x, out, rng.choice(["none", "gelu", "silu"])))
    C = _log(rng, 1, 4096)
    rows = max(1, min(_log(rng, 1, 200704), 12_000_000 // C))
    return _unnamed(_drop("", do, rows, C, x, out, round(rng.uniform(0.0, 0.6), 3),
                          rng.choice(["", "f32", "bf16"])))


def _unnamed(case):
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    s = dict(case)
    train = case["pass"] == "train"
    t_x = TYPES[case["x"]]
    if case["op"] == "gated_delta":
        B, T, Hk, H, Dk, Dv = (case[n] for n in ("B", "T", "Hk", "H", "Dk", "Dv"))
        unit = 1.0 if case["norm"] else 1.0 / math.sqrt(Dk)
        s["q"], s["k"] = (normal(B, T, Hk, Dk) * unit).to(t_x), (normal(B, T, Hk, Dk) * unit).to(t_x)
        s["v"] = normal(B, T, H, Dv).to(t_x)
        # each head has a rate of its own; steps vary from token to token
        rate = torch.exp(uniform(H) * 5.0 - 5.0)
        s["g"] = -rate * torch.log1p(torch.exp(normal(B, T, H)))
        s["beta"] = torch.sigmoid(normal(B, T, H))
        s["state_t"] = 0.3 * normal(B, H, Dk, Dv) if case["state"] else None
        s["next"] = torch.empty(B, H, Dk, Dv, device=DEV) if case["pass"] == "step" else None
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = (uniform(B) * (T + 1)).to(torch.int32).clamp_(max=T)
        s["scale"] = 1.0 / math.sqrt(Dk)
        s["eps"] = QK_EPS if case["norm"] else 0.0
        s["dout"] = normal(B, T, H, Dv).to(t_x) if train else None
        s["dstate"] = 0.1 * normal(B, H, Dk, Dv) if train and case["state"] else None
    elif case["op"] == "group_norm":
        B, S, C = case["B"], case["S"], case["C"]
        # channels with offsets and sizes of their own
        x = normal(B, S, C) * (0.5 + uniform(C)) + 0.5 * normal(C)
        s["x_t"] = x.to(t_x)
        s["gain"], s["bias"] = 1.0 + 0.2 * normal(C), 0.2 * normal(C)
        s["dout"] = (0.05 * normal(B, S, C)).to(TYPES[case["out"]]) if train else None
    else:
        rows, C = case["rows"], case["C"]
        s["x_t"] = normal(rows, C).to(t_x)
        s["res_t"] = normal(rows, C).to(TYPES[case["res"]]) if case["res"] else None
        s["dout"] = normal(rows, C).to(TYPES[case["out"]]) if train else None
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ (seed * 0x10001), 3 + seed
    return s


# -------------------------------------------------------------- plain forms

def _inverse(L):
    """(I + L)^-1 of strictly lower triangular L [..., n, n], row by row."""
    n = L.shape[-1]
    X = torch.eye(n, device=L.device).expand_as(L).clone()
    for i in range(1, n):
        X[..., i, :] -= (L[..., i, :i, None] * X[..., :i, :]).sum(-2)
    return X


def _plain_delta(s):
    B, T, Hk, H, Dk, Dv = (s[n] for n in ("B", "T", "Hk", "H", "Dk", "Dv"))
    n = H // Hk
    C = min(CHUNK, T)
    N = -(-T // C)
    live = torch.ones(B, T, device=DEV, dtype=torch.bool)
    if s["lengths"] is not None:
        live = torch.arange(T, device=DEV)[None] < s["lengths"][:, None]

    def chunks(t):          # [B,T,h,d] -> [B,h,N,C,d] in 32 bits, zero where not live
        t = torch.where(live[:, :, None, None], t.float(), 0.0)
        t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, N * C - T))
        return t.view(B, N, C, t.shape[2], t.shape[3]).permute(0, 3, 1, 2, 4)

    def tokens(t):          # the way back
        return t.permute(0, 2, 3, 1, 4).reshape(B, N * C, t.shape[1], t.shape[4])[:, :T]

    q, k = chunks(s["q"]), chunks(s["k"])
    rq = rk = None
    if s["eps"] > 0:
        rq = (q.square().sum(-1, keepdim=True) + s["eps"]).rsqrt()
        rk = (k.square().sum(-1, keepdim=True) + s["eps"]).rsqrt()
        q, k = q * rq, k * rk
    qn, kn = q, k
    q, k = q.repeat_interleave(n, 1), k.repeat_interleave(n, 1)
    v = chunks(s["v"])
    G = chunks(s["g"][..., None]).cumsum(-2)
    beta = chunks(s["beta"][..., None])
    sc = s["scale"]
    gam, end = G.exp(), (G[..., -1:, :] - G).exp()
    low = torch.ones(C, C, device=DEV, dtype=torch.bool).tril()
    strict = low.tril(-1)
    decay = torch.where(low, (G - G.transpose(-1, -2)).exp(), 0.0)
    M = torch.where(strict, (k @ k.transpose(-1, -2)) * decay, 0.0)
    P = (q @ k.transpose(-1, -2)) * decay
    X = _inverse(M * beta.transpose(-1, -2))
    S = s["state_t"] if s["state_t"] is not None else torch.zeros(B, H, Dk, Dv, device=DEV)
    starts, errs, outs = [], [], []
    for c in range(N):
        e = X[:, :, c] @ (v[:, :, c] - gam[:, :, c] * (k[:, :, c] @ S))
        u = beta[:, :, c] * e
        outs.append(sc * (gam[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ u))
        starts.append(S)
        errs.append(e)
        S = gam[:, :, c, -1:] * S + (k[:, :, c] * end[:, :, c]).transpose(-1, -2) @ u
    t_x = s["q"].dtype
    out = {"out": tokens(torch.stack(outs, 2)).to(t_x), "state": S}
    if s["pass"] != "train":
        return out
    # backward: the states' gradients from the last chunk to the first, then
    # everything else chunk by chunk at once
    do = chunks(s["dout"])
    E, S0 = torch.stack(errs, 2), torch.stack(starts, 2)
    PtDo = sc * (P.transpose(-1, -2) @ do)
    dS = s["dstate"] if s["dstate"] is not None else torch.zeros_like(S)
    ends, dvs, dus = [None] * N, [None] * N, [None] * N
    for c in reversed(range(N)):
        ends[c] = dS
        du = end[:, :, c] * (k[:, :, c] @ dS) + PtDo[:, :, c]
        dv = X[:, :, c].transpose(-1, -2) @ (beta[:, :, c] * du)
        dus[c], dvs[c] = du, dv
        dS = (gam[:, :, c, -1:] * dS + sc * (q[:, :, c] * gam[:, :, c]).transpose(-1, -2) @ do[:, :, c]
              - (k[:, :, c] * gam[:, :, c]).transpose(-1, -2) @ dv)
    D1, dv, du = torch.stack(ends, 2), torch.stack(dvs, 2), torch.stack(dus, 2)
    Et = E.transpose(-1, -2)
    dP = sc * (do @ Et) * beta.transpose(-1, -2)
    dM = torch.where(strict, -(dv @ Et), 0.0)
    wP, wM = torch.where(low, dP * decay, 0.0), dM * beta.transpose(-1, -2) * decay
    rd_q = sc * gam * (do @ S0.transpose(-1, -2))
    rd_k = -gam * (dv @ S0.transpose(-1, -2))
    wr_k = end * beta * (E @ D1.transpose(-1, -2))
    dq = rd_q + wP @ k
    dk = rd_k + wr_k + wP.transpose(-1, -2) @ q + (wM + wM.transpose(-1, -2)) @ k
    dbeta = (E * du).sum(-1, keepdim=True) + (M * dM).sum(-2)[..., None]
    both = P * dP + M * dM * beta.transpose(-1, -2)
    both = torch.where(strict, both, 0.0)
    into = (both.sum(-1) - both.sum(-2))[..., None] + (q * rd_q + k * rd_k).sum(-1, keepdim=True)
    wr = (k * wr_k).sum(-1, keepdim=True)
    dg = into.flip(-2).cumsum(-2).flip(-2) + wr.cumsum(-2) - wr
    dg = dg + (gam[..., -1:, :] * (S0 * D1).sum((-1, -2), keepdim=True))
    dq = dq.view(B, Hk, n, N, C, Dk).sum(2)
    dk = dk.view(B, Hk, n, N, C, Dk).sum(2)
    if rq is not None:
        dq = rq * (dq - qn * (qn * dq).sum(-1, keepdim=True))
        dk = rk * (dk - kn * (kn * dk).sum(-1, keepdim=True))
    keep = live[:, :, None]
    out.update(dq=tokens(dq).to(t_x), dk=tokens(dk).to(t_x), dv=tokens(dv).to(t_x),
               dg=torch.where(keep, tokens(dg)[..., 0], 0.0),
               dbeta=torch.where(keep, tokens(dbeta)[..., 0], 0.0))
    if s["state_t"] is not None:
        out["dstate"] = dS
    return out


def _plain_group_norm(s):
    B, S, C, G, kind = (s[n] for n in ("B", "S", "C", "G", "act"))
    x = s["x_t"].float().view(B, S, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    xc = x - mean
    rstd = (xc.square().mean((1, 3), keepdim=True) + GN_EPS).rsqrt()
    xh = (xc * rstd).view(B, S, C)
    z = xh * s["gain"] + s["bias"]
    cdf = None
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * SQRT_HALF))
    elif kind == "silu":
        cdf = torch.sigmoid(z)
    out = {"y": (z if cdf is None else z * cdf).to(TYPES[s["out"]])}
    if s["pass"] == "fwd":
        return out
    dz = s["dout"].float()
    if kind == "gelu":
        dz = dz * (cdf + z * torch.exp(-0.5 * z * z) * INV_SQRT_2PI)
    elif kind == "silu":
        dz = dz * cdf * (1.0 + z * (1.0 - cdf))
    d = (dz * s["gain"]).view(B, S, G, C // G)
    xg = xh.view(B, S, G, C // G)
    dx = rstd * (d - d.mean((1, 3), keepdim=True) - xg * (d * xg).mean((1, 3), keepdim=True))
    out.update(dx=dx.reshape(B, S, C).to(TYPES[s["x"]]), dgain=(dz * xh).sum((0, 1)),
               dbias=dz.sum((0, 1)))
    return out


def _philox(blocks, seed, offset):
    """Philox4x32-10 of blocks 0 .. blocks-1 as 8 columns of 16 bits."""
    low = 0xFFFFFFFF
    k = torch.arange(blocks, device=DEV, dtype=torch.int64)
    c0, c1 = k & low, k >> 32
    c2, c3 = torch.full_like(k, offset & low), torch.full_like(k, (offset >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        # 64-bit products wrap; their upper words are right after the mask
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & low) ^ c1 ^ k0, p1 & low,
                          ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), 1)
    return torch.stack((words & 0xFFFF, words >> 16), 2).view(blocks, 8)


def _plain_dropout(s):
    x = s["x_t"]
    thr = min(int(math.floor(s["p"] * 65536.0 + 0.5)), 65535)
    bits = _philox(-(-x.numel() // 8), s["seed"], s["offset"])
    keep = (bits.reshape(-1)[:x.numel()] >= thr).view(x.shape)
    up = 65536.0 / (65536.0 - thr)
    y = torch.where(keep, x.float() * up, 0.0)
    if s["res_t"] is not None:
        y = y + s["res_t"].float()
    out = {"y": y.to(TYPES[s["out"]])}
    if s["pass"] == "train":
        out["dx"] = torch.where(keep, s["dout"].float() * up, 0.0).to(x.dtype)
    return out


# ---------------------------------------------------------- the entry points

def _own_delta(s):
    from self_referential_memory_amd import srnl
    kw = {"lengths": s["lengths"], "scale": s["scale"], "norm_eps": s["eps"]}
    q, k, v, g, beta = s["q"], s["k"], s["v"], s["g"], s["beta"]
    if s["pass"] == "step":
        out, state = srnl.gated_delta_step(q, k, v, g, beta, s["state_t"], state_out=s["next"], **kw)
        return {"out": out, "state": state}
    if s["pass"] == "fwd":
        out, state = srnl.gated_delta_fwd(q, k, v, g, beta, state=s["state_t"], **kw)
        return {"out": out, "state": state}
    out, state, record = srnl.gated_delta_fwd(q, k, v, g, beta, state=s["state_t"], record=True, **kw)
    dq, dk, dv, dg, dbeta, dstate = srnl.gated_delta_bwd(
        s["dout"], q, k, v, g, beta, record, state=s["state_t"], dstate=s["dstate"], **kw)
    res = {"out": out, "state": state, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
    if s["state_t"] is not None:
        res["dstate"] = dstate
    return res


def _own_group_norm(s):
    from self_referential_memory_amd import srnl
    x, G, gain, bias, act = s["x_t"], s["G"], s["gain"], s["bias"], s["act"]
    if s["pass"] == "fwd":
        return {"y": srnl.group_norm_fwd(x, G, gain, bias, GN_EPS, act=act, out_dtype=TYPES[s["out"]])}
    y, mean, rstd = srnl.group_norm_fwd(x, G, gain, bias, GN_EPS, act=act,
                                        out_dtype=TYPES[s["out"]], stats=True)
    dx, dgain, dbias = srnl.group_norm_bwd(s["dout"], x, G, gain, bias, mean, rstd, act=act)
    return {"y": y, "dx": dx, "dgain": dgain, "dbias": dbias}


def _own_dropout(s):
    from self_referential_memory_amd import srnl
    x = s["x_t"]
    out = {"y": srnl.dropout_fwd(x, s["p"], s["seed"], s["offset"], residual=s["res_t"],
                                 out_dtype=TYPES[s["out"]])}
    if s["pass"] == "train":
        out["dx"] = srnl.dropout_bwd(s["dout"], s["p"], s["seed"], s["offset"], dtype=x.dtype)
    return out


_PLAIN = {"gated_delta": _plain_delta, "group_norm": _plain_group_norm, "dropout": _plain_dropout}
_OWN = {"gated_delta": _own_delta, "group_norm": _own_group_norm, "dropout": _own_dropout}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    """Inputs read once, outputs written once; for the delta rule the flops of
    its recurrence (the products with the state, its update and its decay)."""
    sx = TYPES[case["x"]].itemsize
    train = case["pass"] == "train"
    if case["op"] == "gated_delta":
        B, T, Hk, H, Dk, Dv = (case[n] for n in ("B", "T", "Hk", "H", "Dk", "Dv"))
        qkv = B * T * (2 * Hk * Dk + H * Dv)
        states = B * H * Dk * Dv * 4
        moved = (qkv + B * T * H * Dv) * sx + B * T * H * 8 + states * (2 if case["state"] else 1)
        flops = 7 * B * T * H * Dk * Dv
        if train:
            moved += (2 * qkv + B * T * H * Dv) * sx + B * T * H * 16
            moved += states * (3 if case["state"] else 0)
            flops += 14 * B * T * H * Dk * Dv
        return {"bytes": moved, "flops": flops}
    so = TYPES[case["out"]].itemsize
    if case["op"] == "group_norm":
        n = case["B"] * case["S"] * case["C"]
        moved, flops = n * (sx + so) + 8 * case["C"], 12 * n
        if train:
            moved, flops = moved + n * (2 * sx + so) + 16 * case["C"], flops + 24 * n
        return {"bytes": moved, "flops": flops}
    n = case["rows"] * case["C"]
    res = TYPES[case["res"]].itemsize if case["res"] else 0
    moved, flops = n * (sx + so + res), 3 * n
    if train:
        moved, flops = moved + n * (sx + so), flops + 2 * n
    return {"bytes": moved, "flops": flops}


# -------------------------------------------------------------------- exact

def _exact_delta(case, s):
    """Token by token in 64 bits; the backward pass steps through the states,
    kept at every 64th token and formed again between."""
    B, T, Hk, H, Dk, Dv = (case[n] for n in ("B", "T", "Hk", "H", "Dk", "Dv"))
    f64 = torch.float64
    n = H // Hk
    raw = {"q": s["q"].double(), "k": s["k"].double()}
    size = {}
    unit = {}
    for name, t in raw.items():
        size[name] = torch.ones(B, T, Hk, 1, device=DEV, dtype=f64)
        if s["eps"] > 0:
            size[name] = torch.sqrt((t * t).sum(-1, keepdim=True) + s["eps"])
        unit[name] = t / size[name]
    head = torch.arange(H, device=DEV) // n
    q, k = unit["q"][:, :, head], unit["k"][:, :, head]
    v, b = s["v"].double(), s["beta"].double()
    a = torch.exp(s["g"].double())
    last = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device=DEV)
    on = (torch.arange(T, device=DEV)[:, None] < last[None]).to(f64)[:, :, None]       # [T,B,1]
    S = torch.zeros(B, H, Dk, Dv, device=DEV, dtype=f64)
    if s["state_t"] is not None:
        S = s["state_t"].double()

    def advance(S, t):
        """The state after token t, with the decayed state and the error."""
        w = on[t][..., None, None]
        A = S * (1 + w * (a[:, t, :, None, None] - 1))
        e = v[:, t] - (A * k[:, t, :, :, None]).sum(2)
        return A + w * k[:, t, :, :, None] * (b[:, t, :, None] * e)[:, :, None], A, e

    y = torch.zeros(B, T, H, Dv, device=DEV, dtype=f64)
    kept = []
    for t in range(T):
        if t % 64 == 0:
            kept.append(S)
        S, _, _ = advance(S, t)
        y[:, t] = s["scale"] * on[t][..., None] * (S * q[:, t, :, :, None]).sum(2)
    out = {"out": y, "state": S}
    if case["pass"] != "train":
        return out
    do = s["dout"].double()
    dq, dk = torch.zeros_like(q), torch.zeros_like(k)
    dv, db, dg = torch.zeros_like(v), torch.zeros_like(b), torch.zeros_like(b)
    W = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    for c in reversed(range(len(kept))):
        part = []
        S = kept[c]
        for t in range(64 * c, min(T, 64 * c + 64)):
            N, A, e = advance(S, t)
            part.append((t, S, A, e, N))
            S = N
        for t, S, A, e, N in reversed(part):
            w = on[t][..., None]
            y_bar = s["scale"] * w * do[:, t]
            dq[:, t] = (N * y_bar[:, :, None]).sum(-1)
            W = W + q[:, t, :, :, None] * y_bar[:, :, None]
            u_bar = w * (W * k[:, t, :, :, None]).sum(2)
            e_bar = b[:, t, :, None] * u_bar
            db[:, t] = (u_bar * e).sum(-1)
            dv[:, t] = e_bar
            dk[:, t] = w * (W * (b[:, t, :, None] * e)[:, :, None]).sum(-1) - (A * e_bar[:, :, None]).sum(-1)
            W = W - k[:, t, :, :, None] * e_bar[:, :, None]
            dg[:, t] = on[t] * (W * A).sum((-1, -2))
            W = W * (1 + on[t][..., None, None] * (a[:, t, :, None, None] - 1))
    grads = {}
    for name, d in (("q", dq), ("k", dk)):
        d = d.view(B, T, Hk, n, Dk).sum(3)
        if s["eps"] > 0:
            d = (d - unit[name] * (unit[name] * d).sum(-1, keepdim=True)) / size[name]
        grads["d" + name] = d
    out.update(dq=grads["dq"], dk=grads["dk"], dv=dv, dg=dg, dbeta=db)
    if s["state_t"] is not None:
        out["dstate"] = W
    return out


def _exact_group_norm(case, s):
    B, S, C, G = case["B"], case["S"], case["C"], case["G"]
    n = S * (C // G)
    # a group's elements as one row
    rows = s["x_t"].double().view(B, S, G, -1).transpose(1, 2).reshape(B * G, n)
    gain = s["gain"].double().view(1, G, 1, -1)
    bias = s["bias"].double().view(1, G, 1, -1)
    var, mean = torch.var_mean(rows, 1, correction=0, keepdim=True)
    size = torch.sqrt(var + GN_EPS)
    h = ((rows - mean) / size).view(B, G, S, -1)
    z = torch.addcmul(bias, h, gain)
    if case["act"] == "gelu":
        cdf = torch.special.erfc(-z / math.sqrt(2.0)) / 2
        slope = cdf + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    elif case["act"] == "silu":
        cdf = (1 + torch.tanh(z / 2)) / 2
        slope = cdf + z * cdf * (1 - cdf)
    else:
        cdf = slope = torch.ones_like(z)

    def back(t):
        return t.view(B, G, S, -1).transpose(1, 2).reshape(B, S, C)

    out = {"y": back(z * cdf)}
    if case["pass"] == "train":
        dz = s["dout"].double().view(B, S, G, -1).transpose(1, 2) * slope
        d, hr = (dz * gain).reshape(B * G, n), h.reshape(B * G, n)
        along = torch.stack((d.sum(1), torch.linalg.vecdot(d, hr)), 1) / n
        out["dx"] = back((d - along[:, :1] - hr * along[:, 1:]) / size)
        out["dgain"] = torch.einsum("bgsc,bgsc->gc", dz, h).reshape(C)
        out["dbias"] = dz.sum((0, 2)).reshape(C)
    return out


def _exact_dropout(case, s):
    m = s["x_t"].numel()
    blocks = np.arange((m + 7) // 8, dtype=np.uint64)
    word = np.uint64(0xFFFFFFFF)
    shift = np.uint64(32)
    ctr = [blocks & word, blocks >> shift, np.full_like(blocks, s["offset"] % 2 ** 32),
           np.full_like(blocks, s["offset"] // 2 ** 32 % 2 ** 32)]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32 % 2 ** 32]
    for r in range(10):
        left, right = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        k0 = np.uint64((key[0] + r * 0x9E3779B9) % 2 ** 32)
        k1 = np.uint64((key[1] + r * 0xBB67AE85) % 2 ** 32)
        ctr = [(right >> shift) ^ ctr[1] ^ k0, right & word, (left >> shift) ^ ctr[3] ^ k1, left & word]
    bits = np.stack(ctr, 1).astype("<u4").view("<u2").reshape(-1)[:m].astype(np.int32)
    cut = min(math.floor(case["p"] * 65536 + 0.5), 65535)
    keep = torch.from_numpy(bits >= cut).to(DEV).view(s["x_t"].shape)
    rate = 1 - cut / 65536

    def thin(t):
        return torch.where(keep, t.double() / rate, torch.zeros((), device=DEV, dtype=torch.float64))

    y = thin(s["x_t"])
    if s["res_t"] is not None:
        y = y + s["res_t"].double()
    return {"y": y, "dx": thin(s["dout"])} if case["pass"] == "train" else {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    f = {"gated_delta": _exact_delta, "group_norm": _exact_group_norm, "dropout": _exact_dropout}
    return f[case["op"]](case, s)
