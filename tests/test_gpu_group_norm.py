"""Group norm with an activation, forward and backward, against its formulas in
float64, element by element.

Bounds, fixed before the first run; u = 2^-24, half a step of fp32. A thread
sums `lane` cells about its first one, then at most 256 lanes and the slabs'
channels join, so a sum's longest chain is `chain` additions: off by at most 2
(chain + 8) u of its terms' magnitudes. The distances from the first cell make
a lane's squares at most 2 (1 + lane) times those about the mean, and its
variance off by that times (lane + 8) u. Activations as the linear layer's: erf's
formula 0.75e-7 |z|, exp and the reciprocal a few u; slopes at most 1.13 in size
and 1.6 in derivative.
"""
import pytest
import torch

from self_referential_memory_amd import srnl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def rnd(seed, *shape, dtype=F32, scale=1.0, offset=0.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + offset).to(DEV).to(dtype)


def within(got, ref, bound, what):
    assert got.shape == ref.shape, what
    over = (got.double() - ref).abs() - (bound + HALF[got.dtype] * ref.abs() + 1e-37)
    assert bool((over <= 0).all()), f"{what}: over by {over.max().item():.3e}"


def act(z, kind):
    """The activation and its slope in float64."""
    if kind == "gelu":
        cdf = torch.special.erfc(-z / 2 ** 0.5) / 2
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    return z, torch.ones_like(z)


def chains(B, S, C, G):
    v = next(n for n in (8, 4, 2, 1) if C % n == 0)
    lanes = max(1, 256 // (C // v))
    items = B * -(-(C // v) // 256)
    slabs = min(-(-1024 // items), -(-S // (8 * lanes)))
    lane = -(-S // (slabs * lanes)) + 8
    return lane, lane + lanes + slabs * (C // G) / 64 + 8


def check(B, S, C, G, x_t, y_t, kind, scale=2.0, offset=3.0):
    x, dout = rnd(C, B, S, C, dtype=x_t, scale=scale, offset=offset), rnd(C + 1, B, S, C, dtype=y_t)
    gain, bias = rnd(C + 2, C, scale=0.3, offset=1.0), rnd(C + 3, C)
    y, mean, rstd = srnl.group_norm_fwd(x, G, gain, bias, 1e-5, act=kind, out_dtype=y_t, stats=True)
    lane, chain = chains(B, S, C, G)

    def grouped(t):
        return t.double().reshape(B, S, G, C // G)

    def over(t):                                     # mean over a group, spread back
        return t.mean((1, 3), keepdim=True)

    def flat(t):
        return t.expand(B, S, G, C // G).reshape(B, S, C)

    X = grouped(x)
    rm = over(X)
    far = (X - rm).abs()
    rr = (over(far.square()) + 1e-5).rsqrt()
    bm = 2 * (chain + 8) * U * (over(far) + far.amax((1, 3), keepdim=True)) + 4 * U * X.abs().amax((1, 3), keepdim=True)
    br = (2 * (1 + lane) * (lane + 8) + 2 * chain) * U + (bm * rr) ** 2
    within(mean, rm[:, 0, :, 0], bm[:, 0, :, 0], "mean")
    within(rstd, rr[:, 0, :, 0], (br * rr)[:, 0, :, 0], "rstd")
    n = flat((X - rm) * rr)
    g64 = gain.double()
    z = n * g64 + bias.double()
    bn = flat(bm * rr + (X - rm).abs() * rr * br) + 4 * U * n.abs() + flat(2 * U * X.abs() * rr)
    bz = bn * g64.abs() + 2 * U * z.abs() + 2 * U * bias.double().abs()
    ry, slope = act(z, kind)
    within(y, ry, 1.13 * bz + (0 if kind == "none" else 2e-5 * ry.abs() + 4e-7 * z.abs()), "y")
    # backward from the exact statistics, rounded to fp32
    mean, rstd = rm[:, 0, :, 0].float(), rr[:, 0, :, 0].float()
    M, R = mean.double()[:, None, :, None], rstd.double()[:, None, :, None]
    n = flat((X - M) * R)
    z = n * g64 + bias.double()
    slope = act(z, kind)[1]
    bn = flat(4 * U * (X - M).abs() * R)
    bz = bn * g64.abs() + 2 * U * (z.abs() + bias.double().abs())
    bs = 0 if kind == "none" else 1.6 * bz + 2e-6 + 1e-6 * z.abs()
    dz = dout.double() * slope
    bdz = dout.double().abs() * bs + 4 * U * dz.abs()
    d, bd = dz * g64, bdz * g64.abs() + 2 * U * (dz * g64).abs()
    dx, dgain, dbias = srnl.group_norm_bwd(dout, x, G, gain, bias, mean, rstd, act=kind)
    k = 2 * (chain + 8) * U
    m1, m2 = over(grouped(d)), over(grouped(d * n))
    b1 = over(grouped(bd)) + k * over(grouped(d.abs()))
    b2 = over(grouped(bd * n.abs() + d.abs() * bn)) + k * over(grouped((d * n).abs()))
    rdx = flat(R) * (d - flat(m1) - n * flat(m2))
    bdx = flat(R) * (bd + flat(b1) + n.abs() * flat(b2) + bn * flat(m2).abs()
                     + 8 * U * (d.abs() + flat(m1).abs() + (n * flat(m2)).abs()))
    within(dx, rdx, bdx, "dx")
    # parameter sums: the slabs and items join 32 at a time
    kp = 2 * (chain + B * 1024 / 32 + 64) * U
    within(dgain, (dz * n).sum((0, 1)), (bdz * n.abs() + dz.abs() * bn + kp * (dz * n).abs()).sum((0, 1)), "dgain")
    within(dbias, dz.sum((0, 1)), (bdz + kp * dz.abs()).sum((0, 1)), "dbias")
    add = rnd(C + 4, B, S, C, dtype=x_t)
    dx2, _, _ = srnl.group_norm_bwd(dout, x, G, gain, bias, mean, rstd, act=kind, dx_add=add, param_grads=False)
    within(dx2, rdx + add.double(), bdx + 4 * U * (rdx.abs() + add.double().abs()), "dx + add")


SIZES = [(1, 1, 8, 8), (1, 1, 1, 1), (2, 1, 24, 3), (3, 7, 10, 5), (1, 49, 512, 32), (2, 196, 256, 16), (2, 63, 210, 7),
         (1, 3136, 64, 16), (3, 5, 4096, 4), (2, 9, 2500, 10), (1, 2000, 3, 1), (2, 33, 20, 20), (70, 17, 36, 6),
         (1, 401, 777, 1), (2, 50, 192, 192),
         # long maps of few items, by slabs: every width of piece
         (1, 9000, 64, 16), (1, 40000, 24, 2), (2, 20011, 20, 4), (1, 30000, 6, 3), (1, 33001, 3, 1), (1, 2000, 4104, 1),
         # many items, by slices: held and read again
         (64, 100, 96, 12), (40, 700, 64, 16), (130, 3000, 12, 3)]


@pytest.mark.parametrize("B,S,C,G", SIZES)
@pytest.mark.parametrize("x_t,y_t", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("kind", ["none", "gelu", "silu"])
def test_forward_and_backward(B, S, C, G, x_t, y_t, kind):
    print("[gnorm]", B, S, C, G, x_t, y_t, kind, flush=True)
    check(B, S, C, G, x_t, y_t, kind)


@pytest.mark.parametrize("B,S,C,G", [
    # slices of 64, 32 and 16 channels, each pass's and type's own
    (64, 196, 256, 16), (64, 784, 128, 16), (300, 100, 64, 8), (64, 1568, 64, 16),
    # few groups of many slabs and channels; few slices, just short and just long enough for slabs
    (3, 2149, 366, 2), (1, 9, 20000, 2), (1, 3584, 256, 32), (1, 3585, 256, 32)])
@pytest.mark.parametrize("x_t,y_t", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_where_a_map_is_cut(B, S, C, G, x_t, y_t):
    print("[gnorm cut]", B, S, C, G, x_t, y_t, flush=True)
    check(B, S, C, G, x_t, y_t, "silu")


def test_constant_maps_and_large_offsets():
    """A constant group has variance 0: y = act(bias). An offset of 1e4 keeps
    its digits. An infinity makes NaN of its item's group alone."""
    x = rnd(1, 4, 300, 64)
    x[0] = 7.3
    x[1] += 1e4
    x[2, 17, 5] = float("inf")
    gain, bias = rnd(2, 64), rnd(3, 64)
    y, mean, rstd = srnl.group_norm_fwd(x, 8, gain, bias, stats=True)
    assert torch.equal(y[0], bias.expand(300, 64))
    X = x.double().reshape(4, 300, 8, 8)
    m = X.mean((1, 3), keepdim=True)
    r = (X.sub(m).square().mean((1, 3), keepdim=True) + 1e-5).rsqrt()
    ref = ((X - m) * r).reshape(4, 300, 64) * gain.double() + bias.double()
    # the mean of values near 1e4 is right to a few steps there, 1e4 2^-24 = 6e-4
    assert (y[1].double() - ref[1]).abs().max() <= 4e-3 * (1 + gain.abs().max().item())
    assert y[2, :, :8].isnan().all() and y[2, :, 8:].isfinite().all() and y[3].isfinite().all()
    clean = x.clone()
    clean[2, 17, 5] = 0.0
    y2 = srnl.group_norm_fwd(clean, 8, gain, bias)
    assert torch.equal(y[:2], y2[:2]) and torch.equal(y[3], y2[3]) and torch.equal(y[2, :, 8:], y2[2, :, 8:])


def test_without_parameters_outputs_not_wanted_and_empty():
    x, dout = rnd(1, 2, 30, 48), rnd(2, 2, 30, 48)
    one, zero = torch.ones(48, device=DEV), torch.zeros(48, device=DEV)
    y, mean, rstd = srnl.group_norm_fwd(x, 6, None, None, act="silu", stats=True)
    assert torch.equal(y, srnl.group_norm_fwd(x, 6, one, zero, act="silu"))
    full = srnl.group_norm_bwd(dout, x, 6, one, zero, mean, rstd, act="silu")
    dx, dg, db = srnl.group_norm_bwd(dout, x, 6, None, None, mean, rstd, act="silu", param_grads=False)
    assert dg is None and db is None and torch.equal(dx, full[0])
    dx, dg, db = srnl.group_norm_bwd(dout, x, 6, None, None, mean, rstd, act="silu", need_dx=False)
    assert dx is None and torch.equal(dg, full[1]) and torch.equal(db, full[2])
    for shape in ((0, 5, 8), (3, 0, 8), (3, 0, 2, 8)):
        e = torch.empty(shape, device=DEV)
        y, mean, rstd = srnl.group_norm_fwd(e, 2, None, None, stats=True)
        assert y.shape == e.shape and not mean.any() and not rstd.any()
        dx, dg, db = srnl.group_norm_bwd(e, e, 2, None, None, mean, rstd)
        assert dx.shape == e.shape and not dg.any() and not db.any()


def test_autograd_matches_differences_and_repeats():
    x, gain, bias = rnd(3, 2, 3, 5, 12, scale=1.5), rnd(4, 12), rnd(5, 12)
    leaves = [t.clone().requires_grad_() for t in (x, gain, bias)]
    w = rnd(6, 2, 3, 5, 12)
    y = srnl.group_norm(leaves[0], 3, leaves[1], leaves[2], act="gelu")
    assert y.shape == x.shape
    grads = torch.autograd.grad((y * w).sum(), leaves)

    def loss(x, gain, bias):
        X = x.reshape(2, 15, 3, 4)
        m = X.mean((1, 3), keepdim=True)
        r = ((X - m).square().mean((1, 3), keepdim=True) + 1e-5).rsqrt()
        z = ((X - m) * r).reshape(2, 3, 5, 12) * gain + bias
        return (act(z, "gelu")[0] * w.double()).sum()

    for i, (t, g) in enumerate(zip((x, gain, bias), grads)):
        v = rnd(7 + i, *t.shape).double()
        h = 1e-5
        args = [a.double() for a in (x, gain, bias)]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        num = ((loss(*up) - loss(*down)) / (2 * h)).item()
        ana = (g.double() * v).sum().item()
        # h^2 of the central difference, and fp32 gradients over at most 360 terms
        assert abs(num - ana) <= 1e-4 * (g.double().norm() * v.norm()).item()
    again = torch.autograd.grad((srnl.group_norm(leaves[0], 3, leaves[1], leaves[2], act="gelu") * w).sum(), leaves)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_other_streams_graphs_and_alignment():
    x, gain, bias = rnd(1, 3, 200, 64), rnd(2, 64), rnd(3, 64)
    dout = rnd(4, 3, 200, 64)

    def both(**kw):
        y, m, r = srnl.group_norm_fwd(x, 8, gain, bias, act="silu", stats=True, **kw)
        return (y, m, r, *srnl.group_norm_bwd(dout, x, 8, gain, bias, m, r, act="silu", **kw))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    long = rnd(5, 1, 9000, 64)
    for src in (x, long):
        with torch.cuda.stream(side):
            srnl.group_norm_fwd(src, 8, gain, bias)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, m, r = srnl.group_norm_fwd(src, 8, gain, bias, act="gelu", stats=True)
            g = srnl.group_norm_bwd(y, src, 8, gain, bias, m, r, act="gelu")
        for seed in range(3):
            src.copy_(rnd(10 + seed, *src.shape))
            graph.replay()
            torch.cuda.synchronize()
            y2, m2, r2 = srnl.group_norm_fwd(src, 8, gain, bias, act="gelu", stats=True)
            g2 = srnl.group_norm_bwd(y2, src, 8, gain, bias, m2, r2, act="gelu")
            assert all(torch.equal(a, b) for a, b in zip((y, *g), (y2, *g2)))
    flat = rnd(6, 3 * 200 * 64 + 1)[1:].view(3, 200, 64)
    with pytest.raises(srnl.SrnlError, match="aligned"):
        srnl.group_norm_fwd(flat, 8, gain, bias)
    with pytest.raises(ValueError, match="contiguous"):
        srnl.group_norm_fwd(x.transpose(1, 2), 8, None, None)
    y = srnl.group_norm(flat.clone().requires_grad_(), 8, gain, bias)
    y.backward(flat)                       # an incoming gradient may start anywhere
