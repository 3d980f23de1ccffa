"""The layers around the operator (layer norm, linear, depthwise 3x3), forward
and backward, against their formulas in float64, element by element.

Bounds, fixed before the first run. u = 2^-24 is half a step of fp32, r(t)
half a step of the output's type relative to the value (bf16 2^-8, fp32
2^-24). A sum of n fp32 terms in any order is off by at most n u times the
sum of the terms' magnitudes when every addition rounds to nearest, twice that
if the matrix unit truncates: bounds are 2 (n + 8) u sum|terms| (the 8 for the
roundings of the terms themselves), carried through the formula, plus r(t)
|y|. An activation adds its own: erf's formula 0.75e-7 |z|, exp and the
reciprocal a few u; its slope is at most 1.13 in size and 1.6 in derivative.
"""
import pytest
import torch

from self_referential_memory_amd import srnl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def say(*a):
    print("[layers]", *a, flush=True)


def rnd(seed, *shape, dtype=F32, scale=1.0, offset=0.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + offset).to(DEV).to(dtype)


def within(got, ref, bound, what):
    """|got - ref| <= bound + half a step of got's type, everywhere."""
    assert got.shape == ref.shape, what
    over = (got.double() - ref).abs() - (bound + HALF[got.dtype] * ref.abs() + 1e-37)
    assert bool((over <= 0).all()), f"{what}: over by {over.max().item():.3e}"


# ------------------------------------------------------------- layer norm

def norm_ref(x, gain, bias, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    var = (x - mean).square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    n = (x - mean) * rstd
    y = n * (1.0 if gain is None else gain.double()) + (0.0 if bias is None else bias.double())
    return y, n, mean, rstd


def norm_bounds(x, n, rstd):
    """Errors of mean (absolute), rstd (relative) and the normalised value."""
    C = x.shape[-1]
    m = 2 * (C + 8) * U * x.double().abs().mean(-1, keepdim=True)
    # (x - mean)^2 summed about the computed mean: its error enters squared
    # (negligible) and through the terms' roundings
    r = 2 * (C + 8) * U + (m * rstd) ** 2
    return m, r, (m + 2 * U * x.double().abs()) * rstd + n.abs() * r + 4 * U * n.abs()


NORM_C = [1, 2, 3, 7, 8, 16, 31, 64, 100, 192, 255, 512, 513, 777, 1024, 1100, 2048, 2500, 4096,
          4097, 5000]


@pytest.mark.parametrize("C", NORM_C)
@pytest.mark.parametrize("x_t,y_t", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
def test_norm_forward_and_backward(C, x_t, y_t):
    rows = 37 if C > 64 else 1031
    say("norm", rows, C, x_t, y_t)
    x = rnd(C, rows, C, dtype=x_t, scale=2.0, offset=3.0)
    gain, bias = rnd(C + 1, C, scale=0.3, offset=1.0), rnd(C + 2, C)
    dout = rnd(C + 3, rows, C, dtype=y_t)
    add = rnd(C + 4, rows, C, dtype=y_t)
    y, mean, rstd = srnl.layer_norm_fwd(x, gain, bias, 1e-5, out_dtype=y_t, stats=True)
    ry, n, rm, rr = norm_ref(x, gain, bias, 1e-5)
    bm, br, bn = norm_bounds(x, n, rr)
    within(mean, rm[:, 0], bm[:, 0], "mean")
    within(rstd, rr[:, 0], (br * rr)[:, 0], "rstd")
    within(y, ry, bn * gain.double().abs() + 2 * U * ry.abs(), "y")
    # the backward pass from the exact statistics, rounded to fp32
    mean, rstd = rm[:, 0].float(), rr[:, 0].float()
    for a in (None, add):
        dx, dgain, dbias = srnl.layer_norm_bwd(dout, x, gain, mean, rstd, dx_add=a)
        nn = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
        g, r = dout.double() * gain.double(), rstd.double()[:, None]
        s1, s2 = g.mean(1, keepdim=True), (g * nn).mean(1, keepdim=True)
        rdx = r * (g - s1 - nn * s2) + (0 if a is None else a.double())
        k = 2 * (C + 8) * U
        bdx = r * (k * g.abs().mean(1, keepdim=True)
                   + nn.abs() * k * (g * nn).abs().mean(1, keepdim=True)
                   + 8 * U * (g.abs() + s1.abs() + (nn * s2).abs())) + 4 * U * rdx.abs()
        # n itself: x - mean and the product round once each
        bdx = bdx + r * 4 * U * ((nn * s2).abs() + nn.abs() * (g * nn).abs().mean(1, keepdim=True))
        within(dx, rdx, bdx, "dx")
        kr = 2 * (rows + 8) * U
        within(dgain, (dout.double() * nn).sum(0), kr * (dout.double() * nn).abs().sum(0), "dgain")
        within(dbias, dout.double().sum(0), kr * dout.double().abs().sum(0), "dbias")


def test_norm_without_parameters_and_outputs_not_wanted():
    x, dout = rnd(1, 50, 96), rnd(2, 50, 96)
    y, mean, rstd = srnl.layer_norm_fwd(x, None, None, 1e-5, stats=True)
    ry, n, _, rr = norm_ref(x, None, None, 1e-5)
    within(y, ry, norm_bounds(x, n, rr)[2], "y")
    dx, dg, db = srnl.layer_norm_bwd(dout, x, None, mean, rstd, param_grads=False)
    assert dg is None and db is None
    full = srnl.layer_norm_bwd(dout, x, torch.ones(96, device=DEV), mean, rstd)
    assert torch.equal(dx, full[0])


@pytest.mark.parametrize("C", [64, 65, 5000])
def test_norm_constant_rows_large_offsets_and_masked_extremes(C):
    """A constant row has variance 0: y = bias, dx finite. An offset of 1e4
    keeps its digits (the variance is taken about the mean). A row with an
    infinity is NaN, and only that row."""
    x = rnd(5, 8, C)
    x[0] = 7.0
    x[1] = x[1] + 1e4
    x[2, C // 2] = float("inf")
    gain, bias = rnd(6, C), rnd(7, C)
    y, mean, rstd = srnl.layer_norm_fwd(x, gain, bias, 1e-5, stats=True)
    assert torch.equal(y[0], bias) and rstd[0].item() == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    ry, n, _, rr = norm_ref(x, gain, bias, 1e-5)
    keep = [0, 1, 3, 4, 5, 6, 7]
    b = norm_bounds(x, n, rr)[2] * gain.double().abs() + 2 * U * ry.abs()
    within(y[keep], ry[keep], b[keep], "y")
    assert torch.isnan(y[2]).all()
    dx, _, _ = srnl.layer_norm_bwd(rnd(8, 8, C), x, gain, mean, rstd, param_grads=False)
    assert torch.isfinite(dx[keep]).all()


@pytest.mark.parametrize("C", [8, 100, 640, 2100])
@pytest.mark.parametrize("rows", [1, 2, 5, 33])
def test_norm_backward_of_few_rows(rows, C):
    """A few rows' parameter gradients come from one block, without a workspace."""
    x, dout, gain = rnd(1, rows, C, dtype=BF16), rnd(2, rows, C), rnd(3, C)
    _, n, rm, rr = norm_ref(x, gain, None, 1e-5)
    mean, rstd = rm[:, 0].float(), rr[:, 0].float()
    _, dg, db = srnl.layer_norm_bwd(dout, x, gain, mean, rstd)
    nn = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    t = dout.double() * nn
    within(dg, t.sum(0), 2 * (rows + 8) * U * t.abs().sum(0), "dgain")
    within(db, dout.double().sum(0), 2 * (rows + 8) * U * dout.double().abs().sum(0), "dbias")


def test_norm_no_rows():
    x = torch.empty(0, 64, device=DEV)
    gain = torch.ones(64, device=DEV)
    y, mean, rstd = srnl.layer_norm_fwd(x, gain, gain, stats=True)
    dx, dg, db = srnl.layer_norm_bwd(x, x, gain, mean, rstd)
    assert y.shape == dx.shape == (0, 64)
    assert not dg.any() and not db.any()


# ------------------------------------------------------------- linear

def act_ref(z, act):
    if act == "gelu":
        return z * torch.special.erfc(-z / 2 ** 0.5) / 2
    return z * torch.sigmoid(z) if act == "silu" else z


def slope_ref(z, act):
    if act == "gelu":
        return torch.special.erfc(-z / 2 ** 0.5) / 2 + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s)) if act == "silu" else torch.ones_like(z)


def check_linear(M, K, N, x_t, w_t, y_t, act="none", bias=True, res=None, add=False, seed=0):
    say("linear", M, K, N, x_t, w_t, y_t, act, bias, res, add)
    s = 100 * seed + M + K + N
    x, w = rnd(s, M, K, dtype=x_t), rnd(s + 1, N, K, dtype=w_t, scale=K ** -0.5)
    b = rnd(s + 2, N) if bias else None
    r = rnd(s + 3, M, N, dtype=res) if res else None
    X, W = x.double(), w.double()
    S = X.abs() @ W.abs().t() + (b.double().abs() if bias else 0)
    z = X @ W.t() + (b.double() if bias else 0)
    bz = 2 * (K + 8) * U * S
    y, pre = srnl.linear_fwd(x, w, b, act=act, residual=r, out_dtype=y_t, keep_pre=True)
    within(pre, z, bz, "pre")
    a = act_ref(z, act)
    # exp(-z^2/2) or exp(-z): the argument's rounding times its size, times z
    ba = 1.13 * bz + (1e-7 * z.abs() + 8 * U * (a.abs() + z.abs() * 4) if act != "none" else 0)
    ry = a + (r.double() if res else 0)
    within(y, ry, ba + 2 * U * ry.abs(), "y")
    assert torch.equal(y, srnl.linear_fwd(x, w, b, act=act, residual=r, out_dtype=y_t))

    dout = rnd(s + 4, M, N, dtype=y_t)
    da = rnd(s + 5, M, K, dtype=x_t) if add else None
    zp = z.float()
    dx, dw, db = srnl.linear_bwd(dout, x, w, zp, act=act, dx_add=da)
    sl = slope_ref(zp.double(), act)
    dz = dout.double() * sl
    bdz = dout.double().abs() * (16 * U * (1 + zp.double().abs()) + 1e-7) if act != "none" else 0 * dz
    rdx = dz @ W + (da.double() if add else 0)
    within(dx, rdx, 2 * (N + 8) * U * (dz.abs() @ W.abs()) + bdz @ W.abs() + 2 * U * rdx.abs(), "dx")
    within(dw, dz.t() @ X, 2 * (M + 8) * U * (dz.abs().t() @ X.abs()) + bdz.t() @ X.abs(), "dw")
    within(db, dz.sum(0), 2 * (M + 8) * U * dz.abs().sum(0) + bdz.sum(0), "db")


TYPES = [(BF16, BF16, BF16), (F32, BF16, F32), (F32, F32, F32), (BF16, F32, F32), (F32, BF16, BF16),
         (BF16, BF16, F32)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (1, 512, 2048), (5, 64, 24), (17, 1, 1), (33, 7, 130),
                                   (49, 2048, 512), (65, 72, 200), (130, 333, 77), (1003, 64, 64),
                                   (300, 1000, 264), (257, 40, 1032), (2100, 256, 512)])
def test_linear_sizes_and_types(M, K, N, types):
    check_linear(M, K, N, *types)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("types", TYPES[:3])
@pytest.mark.parametrize("M,K,N", [(3, 96, 160), (700, 129, 257), (2500, 128, 384)])
def test_linear_epilogues(M, K, N, types, act):
    check_linear(M, K, N, *types, act=act, bias=False, res=BF16, add=True, seed=1)
    check_linear(M, K, N, *types, act=act, bias=True, res=F32, seed=2)


def test_linear_large_tiles_at_the_blocks_own_sizes():
    check_linear(9000, 64, 256, F32, BF16, F32, act="gelu", seed=3)
    check_linear(9000, 256, 64, F32, BF16, F32, res=F32, seed=3)
    check_linear(6272, 768, 192, BF16, BF16, BF16, res=BF16, seed=3)
    check_linear(3136, 512, 2048, F32, BF16, F32, act="gelu", seed=3)


NARROW = [(64, 64), (40, 56), (64, 256), (256, 64), (128, 128), (72, 128), (64, 104), (16, 200), (248, 8)]


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, BF16, F32), (F32, F32, F32), (BF16, F32, F32),
                                   (BF16, BF16, F32), (F32, BF16, BF16)])
@pytest.mark.parametrize("K,N", NARROW)
def test_linear_many_rows_of_narrow_layers(K, N, types, act):
    """65536 rows and a ragged rest: the backward pass that keeps the weights
    in LDS, at every width it has and between them."""
    check_linear(65536 + 1237, K, N, *types, act=act, add=K == 64, bias=True, seed=4)


def test_linear_narrow_backward_repeats_and_matches_its_parts():
    x, w, dout = rnd(1, 70000, 64), rnd(2, 256, 64, dtype=BF16), rnd(3, 70000, 256)
    pre = srnl.linear_fwd(x, w, act="gelu", keep_pre=True)[1]
    dx, dw, db = srnl.linear_bwd(dout, x, w, pre, act="gelu")
    again = srnl.linear_bwd(dout, x, w, pre, act="gelu")
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))
    nb = srnl.linear_bwd(dout, x, w, pre, act="gelu", need_db=False)
    assert nb[2] is None and torch.equal(nb[0], dx) and torch.equal(nb[1], dw)
    # one gradient alone takes the tiled kernels: the same sums in another order
    only = srnl.linear_bwd(dout, x, w, pre, act="gelu", need_dw=False, need_db=False)[0]
    assert (only - dx).abs().max() <= 2 * 264 * 2 * U * (dout.abs().max() * 1.13 * w.float().abs().sum(0).max())


def test_linear_parts_of_the_gradient_and_repeats():
    x, w = rnd(1, 900, 72), rnd(2, 104, 72, dtype=BF16)
    dout = rnd(3, 900, 104)
    dx, dw, db = srnl.linear_bwd(dout, x, w)
    for _ in range(3):
        again = srnl.linear_bwd(dout, x, w)
        assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))
    only, n1, n2 = srnl.linear_bwd(dout, x, w, need_dw=False, need_db=False)
    assert n1 is None and n2 is None and torch.equal(only, dx)
    n1, ow, n2 = srnl.linear_bwd(dout, x, w, need_dx=False, need_db=False)
    assert n1 is None and n2 is None and torch.equal(ow, dw)


def test_linear_no_rows_and_leading_axes():
    w, b = rnd(1, 40, 24), rnd(2, 40)
    y, pre = srnl.linear_fwd(torch.empty(0, 24, device=DEV), w, b, act="gelu", keep_pre=True)
    assert y.shape == pre.shape == (0, 40)
    dx, dw, db = srnl.linear_bwd(y, torch.empty(0, 24, device=DEV), w, pre, act="gelu")
    assert dx.shape == (0, 24) and not dw.any() and not db.any()
    x = rnd(3, 2, 5, 7, 24)
    assert torch.equal(srnl.linear_fwd(x, w, b).view(70, 40), srnl.linear_fwd(x.view(70, 24), w, b))


def test_linear_wide_range_values():
    """Products of fp32 values keep fp32's relative accuracy over its range,
    and a row with a NaN or an infinity leaves the other rows alone."""
    x, w = rnd(1, 200, 96), rnd(2, 160, 96)
    x[::3] *= 1e-30
    w[::5] *= 1e25
    y = srnl.linear_fwd(x, w)
    X, W = x.double(), w.double()
    within(y, X @ W.t(), 2 * 104 * U * (X.abs() @ W.abs().t()), "y")
    bad = x.clone()
    bad[7, 3], bad[150, 95] = float("nan"), float("inf")
    z = srnl.linear_fwd(bad, w)
    keep = torch.ones(200, dtype=torch.bool, device=DEV)
    keep[7] = keep[150] = False
    assert torch.equal(z[keep], y[keep]) and not torch.isfinite(z[~keep]).any()


# ------------------------------------------------------------- depthwise 3x3

def dw_ref(u, w):
    H, W = u.shape[1:3]
    p = torch.nn.functional.pad(u, (0, 0, 1, 1, 1, 1))
    return sum(p[:, a:a + H, e:e + W] * w[:, a, e] for a in range(3) for e in range(3))


@pytest.mark.parametrize("u_t,y_t", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,H,W,C", [(1, 1, 1, 1), (2, 1, 5, 3), (1, 7, 1, 6), (3, 5, 7, 64), (1, 7, 7, 512),
                                     (2, 9, 33, 36), (1, 56, 56, 64), (2, 14, 14, 192), (1, 3, 4, 1030),
                                     (5, 30, 2, 257), (1, 200, 3, 10)])
def test_dwconv(B, H, W, C, u_t, y_t):
    say("dwconv", B, H, W, C, u_t, y_t)
    u, w, b = rnd(1, B, H, W, C, dtype=u_t), rnd(2, C, 3, 3), rnd(3, C)
    a1, a2 = rnd(4, B, H, W, C, dtype=BF16), rnd(5, B, H, W, C)
    ud, wd = u.double(), w.double()
    y0, s0 = dw_ref(ud, wd) + b.double(), dw_ref(ud.abs(), wd.abs()) + b.double().abs()
    within(srnl.dwconv_fwd(u, w, b, out_dtype=y_t), y0, 12 * U * s0, "y")
    y2 = y0 + a1.double() + a2.double()
    got = srnl.dwconv_fwd(u, w, b, a1, a2, out_dtype=y_t)
    within(got, y2, 14 * U * (s0 + a1.double().abs() + a2.double().abs()), "y + adds")
    within(srnl.dwconv_fwd(u, w, None, None, a2, out_dtype=y_t), y0 - b.double() + a2.double(),
           14 * U * (s0 + a2.double().abs()), "one add, no bias")
    dy = rnd(6, B, H, W, C, dtype=y_t)
    du, dw, db = srnl.dwconv_bwd(dy, u, w)
    d = dy.double()
    flip = wd.flip(1, 2)
    within(du, dw_ref(d, flip), 12 * U * dw_ref(d.abs(), flip.abs()), "du")
    n = B * H * W
    up = torch.nn.functional.pad(ud, (0, 0, 1, 1, 1, 1))
    for a in range(3):
        for e in range(3):
            t = up[:, a:a + H, e:e + W] * d
            within(dw[:, a, e], t.sum((0, 1, 2)), (n + 8) * U * t.abs().sum((0, 1, 2)), f"dw {a}{e}")
    within(db, d.sum((0, 1, 2)), (n + 8) * U * d.abs().sum((0, 1, 2)), "db")
    assert torch.equal(du, srnl.dwconv_bwd(dy, u, w, param_grads=False)[0])
    none, dw2, db2 = srnl.dwconv_bwd(dy, u, w, need_du=False)
    assert none is None and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_dwconv_no_cells():
    w = rnd(1, 16, 3, 3)
    u = torch.empty(2, 0, 4, 16, device=DEV)
    assert srnl.dwconv_fwd(u, w, None).shape == u.shape
    du, dw, db = srnl.dwconv_bwd(u, u, w)
    assert du.shape == u.shape and not dw.any() and not db.any()


@pytest.mark.parametrize("M,K,N", [(66773, 64, 64), (1003, 333, 777), (1003, 336, 776), (20, 40, 64)])
def test_linear_bwd_infinite_last_row(M, K, N):
    """An infinity in the last row of bf16 inputs makes its own column of the
    weight gradient infinite and nothing else: rows past the last count as
    nothing, in whichever kernel."""
    x = torch.ones(M, K, device=DEV, dtype=BF16)
    x[-1, 5] = float("inf")
    w = torch.ones(N, K, device=DEV, dtype=BF16)
    dout = torch.ones(M, N, device=DEV, dtype=BF16)
    dx, dw, db = srnl.linear_bwd(dout, x, w)
    assert torch.isposinf(dw[:, 5]).all()
    dw[:, 5] = M
    assert (dw == M).all() and (db == M).all() and (dx == N).all()


def test_dwconv_bwd_very_many_channels():
    """More channels than one launch has columns for in the joining kernel."""
    C = 13_500_000
    u = torch.randn(1, 1, 1, C, device=DEV)
    dy = torch.randn(1, 1, 1, C, device=DEV)
    w = torch.ones(C, 3, 3, device=DEV)
    du, dw, db = srnl.dwconv_bwd(dy, u, w)
    assert torch.equal(du, dy) and torch.equal(db, dy.view(-1))
    assert torch.equal(dw[:, 1, 1], (u * dy).view(-1))
    dw[:, 1, 1] = 0
    assert not dw.any()


def test_layers_refuse_empty_rows():
    with pytest.raises(srnl.SrnlError):
        srnl.layer_norm_fwd(torch.empty(3, 0, device=DEV), None, None)
    with pytest.raises(srnl.SrnlError):
        srnl.linear_fwd(torch.empty(3, 0, device=DEV), torch.empty(4, 0, device=DEV))


@pytest.mark.parametrize("M", [4, 3000])
@pytest.mark.parametrize("e", [-100, -112, -126, -140])
def test_linear_tiny_fp32_operands(M, e):
    """fp32 operands near the bottom of the range: each product to 2^-26 of
    itself or 2^-134 of the other operand, the 64 summed in fp32 (at most 64
    roundings of a sum of positive terms, and the output's)."""
    g = torch.Generator().manual_seed(e * e + M)
    x = ((torch.rand(M, 64, generator=g) + 1).double() * 2.0 ** e).float().to(DEV)
    w = ((torch.rand(96, 64, generator=g) + 1) * 2.0 ** min(120, -e)).to(DEV)
    y = srnl.linear_fwd(x, w)
    want = x.double() @ w.double().t()
    bound = want * (2.0 ** -26 + 65 * 2.0 ** -24) + 2.0 ** -134 * w.double().sum(1)
    assert ((y.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("types", [t for t in TYPES if t[2] == F32])
@pytest.mark.parametrize("M,K,N", [(1, 3, 2), (7, 1, 1), (5, 37, 8201), (16, 264, 4200), (30, 100, 8200), (100, 333, 517),
                                   (260, 40, 400), (640, 261, 515), (300, 600, 1100), (40, 517, 5000)])
def test_linear_few_rows_in_blocks_of_each_shape(M, K, N, types):
    """Blocks of 16 x 16 to 64 x 32 and 32 x 64 outputs, reductions that end
    inside a piece, rows that end inside a block, operands shorter than a piece."""
    check_linear(M, K, N, *types, act="silu", res=F32, seed=3)
