"""The layer operators around the SRNL scan, as calls on the GPU: layer norm,
the linear layer with bias, activation and residual in its epilogue, and the
depthwise 3x3 branch, each forward and backward.

Sizes are those of the residual block at the hierarchical backbone's stages
(64 items of 56x56x64 ... 7x7x512, feed-forward width 4C), of the plain
backbone (32 items of 14x14x192), of a single image, and generic odd ones.

A case is one pass: "fwd" (one forward call), "bwd" (one backward call, with
what the forward kept in hand) or "step" (a forward that keeps what the
backward needs, then the backward). ``run`` computes it either with elementary
torch operations in 32 bits, rounded once at the end, or (``own``) with the
package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
SQRT_HALF = math.sqrt(0.5)
INV_SQRT_2PI = 1.0 / math.sqrt(2.0 * math.pi)


# ------------------------------------------------------------------- cases

def _ln(name, do, rows, C, x, out, add=False):
    return {"name": name, "op": "layer_norm", "pass": do, "rows": rows, "C": C, "x": x,
            "out": out, "add": add}


def _lin(name, do, M, K, N, x, w, out, act="none", bias=True, res="", add=False):
    return {"name": name, "op": "linear", "pass": do, "M": M, "K": K, "N": N, "x": x, "w": w,
            "out": out, "act": act, "bias": bias, "res": res, "add": add}


def _dw(name, do, B, H, W, C, x, out, adds=0):
    return {"name": name, "op": "dwconv", "pass": do, "B": B, "H": H, "W": W, "C": C, "x": x,
            "out": out, "adds": adds}


def listed():
    return [
        # inference norm over the last stage's map, 64 items of 7x7
        _ln("norm_stage4_fwd", "fwd", 3136, 512, "bf16", "bf16"),
        # the block's first norm in training at stage 1: x in bf16, the norm's
        # output and its gradient in fp32, the residual's gradient added
        _ln("norm_stage1_bwd", "bwd", 200704, 64, "bf16", "f32", add=True),
        # a generic odd width, one training step
        _ln("norm_odd_step", "step", 12001, 777, "bf16", "bf16"),
        # one token through the last stage's first feed-forward product
        _lin("ffn_up_token", "fwd", 1, 512, 2048, "bf16", "bf16", "bf16", act="gelu"),
        # one image's last-stage map (7x7) through the second product
        _lin("ffn_down_image", "fwd", 49, 2048, 512, "bf16", "bf16", "bf16", res="bf16"),
        # the first feed-forward product of a stage-1 training step
        _lin("ffn_up_stage1", "fwd", 200704, 64, 256, "f32", "bf16", "f32", act="gelu"),
        # ... and its backward pass
        _lin("ffn_up_stage1_bwd", "bwd", 200704, 64, 256, "f32", "bf16", "f32", act="gelu"),
        # the second feed-forward product of the plain backbone, forward and
        # backward, bf16 activations
        _lin("ffn_down_plain_step", "step", 6272, 768, 192, "bf16", "bf16", "bf16", res="bf16"),
        # fp32 activations and weights, every size odd
        _lin("odd_f32_step", "step", 1003, 333, 777, "f32", "f32", "f32", act="silu"),
        # a wide projection over a long batch
        _lin("wide_fwd", "fwd", 16384, 2048, 2048, "bf16", "bf16", "bf16"),
        # one image's last-stage map through the depthwise branch
        _dw("dwconv_image", "fwd", 1, 7, 7, 512, "bf16", "bf16", adds=2),
        # the depthwise branch's backward pass at stage 1
        _dw("dwconv_stage1_bwd", "bwd", 64, 56, 56, 64, "f32", "f32"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, v))
    r = rng.random()
    if r < 0.35 and v >= 64:
        return v // 32 * 32          # widths are mostly multiples of 32 ...
    if r < 0.5 and v >= 16:
        return v // 8 * 8            # ... or of 8
    return v                         # and sometimes anything


def draw(rng):
    op = rng.choice(["layer_norm", "linear", "linear", "dwconv"])
    do = rng.choice(["fwd", "bwd", "step"])
    x, out = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    if op == "layer_norm":
        C = _log(rng, 16, 4096)
        rows = min(_log(rng, 1, 200704), 12_000_000 // C)
        return _unnamed(_ln("", do, rows, C, x, out, add=do != "fwd" and rng.random() < 0.5))
    if op == "linear":
        K, N = _log(rng, 16, 2048), _log(rng, 16, 2048)
        M = _log(rng, 1, 200704)
        M = max(1, min(M, 60_000_000 // (K + N), 8_000_000_000 // (K * N)))
        act = rng.choice(["none", "gelu", "silu"])
        return _unnamed(_lin("", do, M, K, N, x, rng.choice(["f32", "bf16"]), out, act=act,
                             bias=rng.random() < 0.8, res=rng.choice(["", "f32", "bf16"]),
                             add=do != "fwd" and rng.random() < 0.3))
    B, C = _log(rng, 1, 64), _log(rng, 16, 512)
    side = max(3, int(math.sqrt(12_000_000 / (B * C))))
    H, W = min(_log(rng, 3, 200), side), min(_log(rng, 3, 304), side)
    return _unnamed(_dw("", do, B, H, W, C, x, out, adds=rng.choice([0, 1, 2]) if do != "bwd" else 0))


def _unnamed(case):
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    """Inputs on the GPU, made from the seed alone: activations of a network
    (unit scale, an offset and a scale per channel, the odd large token),
    weights of scale 1/sqrt(fan in), small gradients; for a backward pass also
    what the forward kept."""
    gen = torch.Generator(DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=gen)

    def act(rows, C):
        v = normal(rows, C) * (0.5 + normal(C).abs()) + 0.5 * normal(C)
        return v * (1.0 + 4.0 * (normal(rows, 1) > 2.5))

    s = dict(case)
    t_x, t_out = TYPES[case["x"]], TYPES[case["out"]]
    grads = case["pass"] != "fwd"
    if case["op"] == "layer_norm":
        rows, C = case["rows"], case["C"]
        s["x_t"] = act(rows, C).to(t_x)
        s["gain"], s["bias_t"] = 1.0 + 0.2 * normal(C), 0.2 * normal(C)
        s["dout"] = (0.05 * normal(rows, C)).to(t_out) if grads else None
        s["add_t"] = 0.05 * normal(rows, C) if case["add"] else None
        if case["pass"] == "bwd":
            xf = s["x_t"].double()
            mean = xf.mean(1)
            var = (xf - mean[:, None]).square().mean(1)
            s["mean"], s["rstd"] = mean.float(), (var + EPS).rsqrt().float()
    elif case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x_t"] = act(M, K).to(t_x)
        s["w_t"] = (normal(N, K) / math.sqrt(K)).to(TYPES[case["w"]])
        s["bias_t"] = 0.2 * normal(N) if case["bias"] else None
        s["res_t"] = normal(M, N).to(TYPES[case["res"]]) if case["res"] and case["pass"] != "bwd" else None
        s["dout"] = (0.05 * normal(M, N)).to(t_out) if grads else None
        s["add_t"] = (0.05 * normal(M, K)).to(t_x) if case["add"] else None
        s["pre"] = None
        if case["pass"] == "bwd" and case["act"] != "none":
            z = s["x_t"].float() @ s["w_t"].float().t()
            s["pre"] = z + s["bias_t"] if case["bias"] else z
    else:
        B, H, W, C = case["B"], case["H"], case["W"], case["C"]
        cells = B * H * W
        s["x_t"] = act(cells, C).to(t_x).view(B, H, W, C)
        s["w_t"], s["bias_t"] = normal(C, 3, 3) / 3.0, 0.2 * normal(C)
        s["adds_t"] = [normal(B, H, W, C).to(t_out) for _ in range(case["adds"])]
        s["dout"] = (0.05 * normal(B, H, W, C)).to(t_out) if grads else None
    return s


# -------------------------------------------------------------- plain forms

def _plain_layer_norm(s):
    x = s["x_t"].float()
    y = None
    if s["pass"] == "bwd":
        mean, rstd = s["mean"][:, None], s["rstd"][:, None]
        xh = (x - mean) * rstd
    else:
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + EPS).rsqrt()
        xh = xc * rstd
        y = (xh * s["gain"] + s["bias_t"]).to(TYPES[s["out"]])
        if s["pass"] == "fwd":
            return {"y": y}
    dy = s["dout"].float()
    g = dy * s["gain"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["add_t"] is not None:
        dx = dx + s["add_t"]
    grads = {"dx": dx.to(TYPES[s["x"]]), "dgain": (dy * xh).sum(0), "dbias": dy.sum(0)}
    return grads if y is None else {"y": y, **grads}


def _act(z, kind):
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * SQRT_HALF))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_slope(z, kind):
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * SQRT_HALF)) + z * torch.exp(-0.5 * z * z) * INV_SQRT_2PI
    sg = torch.sigmoid(z)
    return sg * (1.0 + z * (1.0 - sg))


def _plain_linear(s):
    x, w, kind = s["x_t"].float(), s["w_t"].float(), s["act"]
    out = {}
    z = s["pre"]
    if s["pass"] != "bwd":
        z = x @ w.t()
        if s["bias_t"] is not None:
            z = z + s["bias_t"]
        y = _act(z, kind)
        if s["res_t"] is not None:
            y = y + s["res_t"].float()
        out["y"] = y.to(TYPES[s["out"]])
        if s["pass"] == "fwd":
            return out
    dz = s["dout"].float()
    if kind != "none":
        dz = dz * _act_slope(z, kind)
    dx = dz @ w
    if s["add_t"] is not None:
        dx = dx + s["add_t"].float()
    out["dx"] = dx.to(TYPES[s["x"]])
    out["dw"] = dz.t() @ x
    if s["bias_t"] is not None:
        out["db"] = dz.sum(0)
    return out


def _windows(v):
    """[B,H,W,C] -> the zero-padded 3x3 neighbourhoods [B,H,W,C,3,3]."""
    p = torch.nn.functional.pad(v, (0, 0, 1, 1, 1, 1))
    return p.unfold(1, 3, 1).unfold(2, 3, 1)


def _plain_dwconv(s):
    u, w = s["x_t"].float(), s["w_t"]
    out = {}
    if s["pass"] != "bwd":
        y = (_windows(u) * w).sum((-1, -2)) + s["bias_t"]
        if len(s["adds_t"]) > 0:
            y = y + s["adds_t"][0].float()
        if len(s["adds_t"]) > 1:
            y = y + s["adds_t"][1].float()
        out["y"] = y.to(TYPES[s["out"]])
        if s["pass"] == "fwd":
            return out
    dy = s["dout"].float()
    near = _windows(dy)
    out["du"] = (near * w.flip(1, 2)).sum((-1, -2)).to(TYPES[s["x"]])
    out["dw"] = (near * u[..., None, None]).sum((0, 1, 2)).flip(1, 2)
    out["db"] = dy.sum((0, 1, 2))
    return out


# ---------------------------------------------------------- the entry points

def _own_layer_norm(s):
    from self_referential_memory_amd import srnl
    mean, rstd = s.get("mean"), s.get("rstd")
    out = {}
    if s["pass"] != "bwd":
        y = srnl.layer_norm_fwd(s["x_t"], s["gain"], s["bias_t"], EPS, out_dtype=TYPES[s["out"]],
                                stats=s["pass"] == "step")
        if s["pass"] == "fwd":
            return {"y": y}
        out["y"], mean, rstd = y
    out["dx"], out["dgain"], out["dbias"] = srnl.layer_norm_bwd(
        s["dout"], s["x_t"], s["gain"], mean, rstd, dx_add=s["add_t"])
    return out


def _own_linear(s):
    from self_referential_memory_amd import srnl
    pre, out = s["pre"], {}
    if s["pass"] != "bwd":
        keep = s["pass"] == "step" and s["act"] != "none"
        y = srnl.linear_fwd(s["x_t"], s["w_t"], s["bias_t"], act=s["act"], residual=s["res_t"],
                            out_dtype=TYPES[s["out"]], keep_pre=keep)
        if keep:
            y, pre = y
        out["y"] = y
        if s["pass"] == "fwd":
            return out
    dx, dw, db = srnl.linear_bwd(s["dout"], s["x_t"], s["w_t"], pre, act=s["act"],
                                 dx_add=s["add_t"], need_db=s["bias_t"] is not None)
    out["dx"], out["dw"] = dx, dw
    if db is not None:
        out["db"] = db
    return out


def _own_dwconv(s):
    from self_referential_memory_amd import srnl
    out = {}
    if s["pass"] != "bwd":
        out["y"] = srnl.dwconv_fwd(s["x_t"], s["w_t"], s["bias_t"], *s["adds_t"],
                                   out_dtype=TYPES[s["out"]])
        if s["pass"] == "fwd":
            return out
    out["du"], out["dw"], out["db"] = srnl.dwconv_bwd(s["dout"], s["x_t"], s["w_t"])
    return out


_PLAIN = {"layer_norm": _plain_layer_norm, "linear": _plain_linear, "dwconv": _plain_dwconv}
_OWN = {"layer_norm": _own_layer_norm, "linear": _own_linear, "dwconv": _own_dwconv}


def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------- work, 64 bits

def work(case):
    """Every input read once, every output written once, and the operator's
    own operations (a multiply-add counts two)."""
    size = {"f32": 4, "bf16": 2}
    sx, so = size[case["x"]], size[case["out"]]
    do = case["pass"]
    fwd, bwd = do != "bwd", do != "fwd"
    if case["op"] == "layer_norm":
        n, C = case["rows"] * case["C"], case["C"]
        by = n * sx + 2 * C * 4 * (1 + bwd)
        by += n * so * (fwd + bwd) + (n * sx if bwd else 0)
        by += (n * 4 if case["add"] else 0) + (8 * case["rows"] if do == "bwd" else 0)
        return {"bytes": by, "flops": n * (8 * fwd + 14 * bwd)}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        by = M * K * sx + N * K * size[case["w"]] + (4 * N if case["bias"] else 0)
        if fwd:
            by += M * N * so + (M * N * size[case["res"]] if case["res"] else 0)
        if bwd:
            by += M * N * so + M * K * sx + N * K * 4 + (4 * N if case["bias"] else 0)
            by += M * K * sx if case["add"] else 0
        if do == "bwd" and case["act"] != "none":
            by += 4 * M * N
        return {"bytes": by, "flops": 2 * M * K * N * (fwd + 2 * bwd)}
    n, C = case["B"] * case["H"] * case["W"] * case["C"], case["C"]
    by = n * sx + 40 * C * (1 + bwd)
    by += n * so * (1 + case["adds"]) if fwd else 0
    by += n * (so + sx) if bwd else 0
    return {"bytes": by, "flops": n * (18 * fwd + 37 * bwd)}


def exact(case, seed):
    """The definitions in 64 bits, term by term and apart from the plain
    forms: the norm's Jacobian applied as a projection, the products through
    addmm, the convolution as nine shifted products. What a backward pass is
    handed (statistics, pre-activations) is an input as it stands."""
    s = prepare(case, seed)
    d = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    fwd, bwd = case["pass"] != "bwd", case["pass"] != "fwd"
    out = {}
    if case["op"] == "layer_norm":
        x, C = d["x_t"], case["C"]
        if case["pass"] == "bwd":
            mu, r = d["mean"].unsqueeze(1), d["rstd"].unsqueeze(1)
        else:
            mu = x.sum(1, keepdim=True) / C
            r = 1.0 / torch.sqrt(((x - mu) ** 2).sum(1, keepdim=True) / C + EPS)
        n = (x - mu) * r
        if fwd:
            out["y"] = torch.addcmul(d["bias_t"], n, d["gain"])
        if bwd:
            g = d["dout"] * d["gain"]
            along = torch.stack([g.sum(1), (g * n).sum(1)], 1) / C
            dx = (g - along[:, :1] - n * along[:, 1:]) * r
            out["dx"] = dx if d["add_t"] is None else dx + d["add_t"]
            out["dgain"] = torch.einsum("rc,rc->c", d["dout"], n)
            out["dbias"] = torch.ones(1, case["rows"], device=DEV, dtype=torch.float64).mm(d["dout"])[0]
        return out
    if case["op"] == "linear":
        x, w, kind = d["x_t"], d["w_t"], case["act"]
        z = d["pre"]
        if z is None:
            b = d["bias_t"] if d["bias_t"] is not None else torch.zeros(case["N"], device=DEV, dtype=torch.float64)
            z = torch.addmm(b, x, w.t())
        # Phi(z) = erfc(-z / sqrt 2) / 2; the logistic function from tanh
        cdf = torch.special.erfc(-z / math.sqrt(2.0)) / 2 if kind == "gelu" else (1 + torch.tanh(z / 2)) / 2
        if fwd:
            y = z if kind == "none" else z * cdf
            out["y"] = y if d["res_t"] is None else y + d["res_t"]
        if bwd:
            dz = d["dout"]
            if kind == "gelu":
                dz = dz * (cdf + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi))
            elif kind == "silu":
                dz = dz * (cdf + z * cdf * (1 - cdf))
            dx = dz.mm(w)
            out["dx"] = dx if d["add_t"] is None else dx + d["add_t"]
            out["dw"] = x.t().mm(dz).t()
            if d["bias_t"] is not None:
                out["db"] = torch.ones(1, case["M"], device=DEV, dtype=torch.float64).mm(dz)[0]
        return out
    H, W, C = case["H"], case["W"], case["C"]
    u, w = d["x_t"], d["w_t"]
    taps = [(a, e) for a in range(3) for e in range(3)]

    def cut(off, n):       # cells p with p + off inside, and where they read
        return slice(max(0, -off), n - max(0, off)), slice(max(0, off), n + min(0, off))

    if fwd:
        y = d["bias_t"].expand_as(u).clone()
        for a, e in taps:
            (i, si), (j, sj) = cut(a - 1, H), cut(e - 1, W)
            y[:, i, j] += u[:, si, sj] * w[:, a, e]
        for t in s["adds_t"]:
            y += t.double()
        out["y"] = y
    if bwd:
        dy, du, dw = d["dout"], torch.zeros_like(u), torch.zeros_like(w)
        for a, e in taps:
            (i, si), (j, sj) = cut(a - 1, H), cut(e - 1, W)
            du[:, si, sj] += dy[:, i, j] * w[:, a, e]
            dw[:, a, e] = (dy[:, i, j] * u[:, si, sj]).reshape(-1, C).sum(0)
        out["du"], out["dw"], out["db"] = du, dw, dy.reshape(-1, C).sum(0)
    return out
