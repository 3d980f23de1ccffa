"""The layers' corners, against their formulas in float64: operands shorter
than one wide load, activations over their whole range. Bounds as derived in
test_gpu_layers.py; an activation's are given with its test."""
import ctypes

import pytest
import torch

from self_referential_memory_amd import srnl
from test_gpu_layers import BF16, DEV, F32, U, act_ref, rnd, say, slope_ref, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x_t,w_t", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_linear_operands_shorter_than_a_load(x_t, w_t):
    """Every product whose operands have one to seven elements, and one side
    short while the other is not: a piece of eight is read elsewhere then, and
    counts as nothing."""
    say("short operands", x_t, w_t)
    for M, K, N in [(m, k, n) for k in range(1, 8) for m in (1, 2, 3, 7, 40) for n in (1, 2, 7, 33)]:
        x, w, b = rnd(M + K, M, K, dtype=x_t), rnd(N + K, N, K, dtype=w_t), rnd(3, N)
        X, W = x.double(), w.double()
        within(srnl.linear_fwd(x, w, b, out_dtype=F32), X @ W.t() + b.double(),
               2 * (K + 8) * U * (X.abs() @ W.abs().t() + b.double().abs()), f"{M} {K} {N}")


# ------------------------------------------------------------- activations

def tail_error(z):
    """Relative error of q = 1 - Phi(|z|) = exp(-z^2/2) P(s), s = |z| / (|z| + 3).

    P: the polynomial's own error, then Horner's seven fused steps (7 u times
    the sum of its terms' magnitudes over P, at most 2 + 6 |z|) and s, which
    is off by 4 u (reciprocal 2 u, sum and product u each) and enters 5.3
    times at most. exp: the argument z^2/2 is off by 3 u of itself (its
    constant and two products), the instruction 2 u; the last product u."""
    a = z.abs()
    fit = torch.where(a < 3, 1.8e-7, torch.where(a < 5, 1.2e-6, 4.2e-6))
    return fit + U * (7 * (2 + 6 * a) + 4 * 5.3 + 1.5 * a * a + 3)


def act_error(z, act):
    if act == "silu":       # exp(-z): its argument is off by 1.5 u of itself, exp 2 u; sum, reciprocal, product
        return ((1.5 * z.abs() + 2) * torch.sigmoid(-z) + 6) * U * act_ref(z, act).abs()
    q = torch.special.erfc(z.abs() / 2 ** 0.5) / 2
    return z.abs() * q * tail_error(z) + 2 * U * act_ref(z, act).abs()


def slope_error(z, act):
    s = torch.sigmoid(z)
    if act == "silu":       # s (1 + z (1 - s)), 1 - s formed from s
        return s * ((1.5 * z.abs() + 8) * U * (1 + 2 * z.abs()) + 4 * U * (1 + z.abs()))
    q = torch.special.erfc(z.abs() / 2 ** 0.5) / 2
    peak = z.abs() * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    return q * tail_error(z) + peak * U * (1.5 * z * z + 6) + 2 * U * (slope_ref(z, act).abs() + 1)


def sweep(n):
    """n values over [-13, 13], every second one within 1.5 of zero."""
    z = torch.linspace(-13, 13, n, dtype=torch.float64)
    z[::2] = torch.linspace(-1.5, 1.5, len(z[::2]), dtype=torch.float64)
    return z.float().to(DEV)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("y_t", [F32, BF16])
@pytest.mark.parametrize("M", [3001, 20001, 60001])
def test_linear_activation_over_its_range(M, y_t, act):
    """z passes through the product unchanged (one weight of 1, the rest 0),
    in the few-rows kernel and both tile sizes; below zero the output keeps
    its own digits, not only the largest value's."""
    say("activation", M, y_t, act)
    z = sweep(M)
    x, w = torch.zeros(M, 8, device=DEV), torch.zeros(16, 8, device=DEV)
    x[:, 0], w[:, 0] = z, 1.0
    y, pre = srnl.linear_fwd(x, w, act=act, out_dtype=y_t, keep_pre=True)
    assert torch.equal(pre, z[:, None].expand(M, 16))
    z = z.double()[:, None].expand(M, 16)
    within(y, act_ref(z, act), act_error(z, act), act)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("y_t", [F32, BF16])
@pytest.mark.parametrize("M", [500, 9000, 70000])
def test_linear_slope_over_its_range(M, y_t, act):
    """dz = act'(z) comes back as dx through a weight of ones on the diagonal:
    formed while staged (with its own pass, and in the narrow form)."""
    say("slope", M, y_t, act)
    N = 8 if M != 9000 else 264                # 264: a pass of its own makes dz
    z = sweep(M * N).view(M, N)
    w = torch.eye(N, device=DEV)
    x = torch.zeros(M, N, device=DEV)
    dx, dw, db = srnl.linear_bwd(torch.ones(M, N, device=DEV, dtype=y_t), x, w, z, act=act)
    z = z.double()
    within(dx, slope_ref(z, act), slope_error(z, act), act)
    assert not dw.any()


def test_linear_activation_of_extremes():
    """z Phi(z) and z logistic(z) as they are in fp32: +infinity stays, the
    largest values stay or vanish, -infinity x 0 and NaN are NaN."""
    v = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 3e38, -3e38, 1e-38, -1e-38,
                      100.0, -100.0, 13.5, -13.5, 15.0, -15.0, 1.0], device=DEV)
    x, w = torch.zeros(16, 8, device=DEV, dtype=BF16), torch.zeros(16, 8, device=DEV, dtype=BF16)
    x[:, 0], w[:, 0] = v.to(BF16), 1.0
    for act in ("gelu", "silu"):
        y = srnl.linear_fwd(x, w, act=act, out_dtype=F32)[:, 0]
        z = x[:, 0].double()
        assert torch.isposinf(y[0]) and torch.isnan(y[1]) and torch.isnan(y[2]), act
        within(y[3:], act_ref(z[3:], act), act_error(z[3:], act) + 2e-36, act)


# ----------------------------------------------------------- depthwise 3x3

def dw_terms(u, w, dy):
    """du, dw, db and the sums of their terms' magnitudes, over the pairs of
    cells that exist: no product with a zero in place of a missing cell."""
    H, W = u.shape[1:3]
    cut = lambda o, n: (slice(max(0, -o), n - max(0, o)), slice(max(0, o), n + min(0, o)))
    du, sdu = torch.zeros_like(dy), torch.zeros_like(dy)
    dw, sdw = torch.zeros_like(w), torch.zeros_like(w)
    for a in range(3):
        for e in range(3):
            (i, si), (j, sj) = cut(a - 1, H), cut(e - 1, W)
            t = dy[:, i, j] * w[:, a, e]
            du[:, si, sj] += t
            sdu[:, si, sj] += t.abs()
            t = dy[:, i, j] * u[:, si, sj]
            dw[:, a, e], sdw[:, a, e] = t.sum((0, 1, 2)), t.abs().sum((0, 1, 2))
    return (du, sdu), (dw, sdw), (dy.sum((0, 1, 2)), dy.abs().sum((0, 1, 2)))


@pytest.mark.parametrize("u_t,y_t", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,H,W,C", [(3, 5, 7, 64), (2, 9, 3, 33), (90, 57, 7, 64), (1, 1, 1, 6), (1, 2, 2, 8),
                                     (600, 11, 5, 24)])
def test_dwconv_bwd_infinities_stay_with_their_terms(B, H, W, C, u_t, y_t):
    """An infinity of u or dy in a channel, at the grid's corners and edges and
    at rows where one block's walk ends: gradients that have it as a term are
    infinite (NaN for opposite ones), the others are finite and right."""
    say("dwconv infinities", B, H, W, C, u_t, y_t)
    g = torch.Generator().manual_seed(B + C)
    u, w, dy = rnd(1, B, H, W, C, dtype=u_t), rnd(2, C, 3, 3), rnd(3, B, H, W, C, dtype=y_t)
    rows = [0, H - 1, 0, H - 1, *torch.randint(H, (C,), generator=g).tolist()]
    cols = [0, W - 1, W // 2, 0, *torch.randint(W, (C,), generator=g).tolist()]
    for c in range(C):
        t = (u, dy)[c % 2]
        t[c % B, rows[c // 2], cols[c // 2], c] = float("-inf" if c % 3 else "inf")
    (rdu, sdu), (rdw, sdw), (rdb, sdb) = dw_terms(u.double(), w.double(), dy.double())
    n = B * H * W
    for got, ref, size, k, what in zip(srnl.dwconv_bwd(dy, u, w), (rdu, rdw, rdb), (sdu, sdw, sdb), (12, n + 8, n + 8),
                                       ("du", "dw", "db")):
        fin = torch.isfinite(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
        assert torch.equal(got[~fin & ~torch.isnan(ref)].double(), ref[~fin & ~torch.isnan(ref)]), what
        within(got[fin], ref[fin], k * U * size[fin], what)


# ----------------------------------------------------- infinities in linear

@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, BF16, F32), (F32, F32, F32), (BF16, F32, F32),
                                   (BF16, BF16, F32)])
@pytest.mark.parametrize("M,K,N", [(20, 40, 64), (300, 7, 5), (1003, 333, 777), (9000, 512, 640), (66773, 64, 64)])
def test_linear_infinities_stay_in_their_rows(M, K, N, types):
    """Whatever an infinity becomes beside fp32 operands, it touches only the
    outputs that have it as a term; those are not finite. Every other output
    is bitwise the one without it."""
    say("linear infinities", M, K, N, types)
    x_t, w_t, y_t = types
    clean = rnd(1, M, K, dtype=x_t), rnd(2, N, K, dtype=w_t), rnd(3, M, N, dtype=y_t)
    x, w, dy = (t.clone() for t in clean)
    m, k, n = M - 1, K // 2, N - 2

    def same(got, want, touched, what):
        assert torch.equal(got[~touched], want[~touched]), what
        assert not torch.isfinite(got[touched]).any(), what

    def lines(shape, *places):
        hit = torch.zeros(shape, dtype=torch.bool, device=DEV)
        for p in places:
            hit[p] = True
        return hit

    every = slice(None)
    y, (dx, dw, db) = srnl.linear_fwd(x, w, out_dtype=y_t), srnl.linear_bwd(dy, x, w)
    x[m, k] = float("inf")
    same(srnl.linear_fwd(x, w, out_dtype=y_t), y, lines((M, N), m), "y of x")
    g = srnl.linear_bwd(dy, x, w)
    assert torch.equal(g[0], dx) and torch.equal(g[2], db)
    same(g[1], dw, lines((N, K), (every, k)), "dw of x")
    x = clean[0]
    w[n, k] = float("-inf")
    same(srnl.linear_fwd(x, w, out_dtype=y_t), y, lines((M, N), (every, n)), "y of w")
    g = srnl.linear_bwd(dy, x, w)
    assert torch.equal(g[1], dw) and torch.equal(g[2], db)
    same(g[0], dx, lines((M, K), (every, k)), "dx of w")
    w = clean[1]
    dy[m, n] = float("inf")
    g = srnl.linear_bwd(dy, x, w)
    same(g[0], dx, lines((M, K), m), "dx of dy")
    same(g[1], dw, lines((N, K), n), "dw of dy")
    same(g[2], db, lines((N,), n), "db of dy")


# ------------------------------------------------------------------ in place

def abi_linear_bwd(dout, x, w, add, dx):
    """srnl_linear_bwd with dx at a given address (the binding makes its own)."""
    L, (N, K), M = srnl.lib(), w.shape, x.shape[0]
    p = srnl.LinearParams(w.data_ptr(), None, None, srnl._dtype_code(x), srnl._dtype_code(w), 0,
                          srnl._dtype_code(dout), 0, torch.cuda.current_stream().cuda_stream)
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(max(16, L.srnl_linear_bwd_workspace_bytes(M, K, N, ctypes.byref(p))), dtype=torch.uint8,
                     device=DEV)
    assert L.srnl_linear_bwd(dout.data_ptr(), x.data_ptr(), M, K, N, ctypes.byref(p), None, add.data_ptr(),
                             dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel()) == 0
    return dw, db


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("C", [5, 8, 12, 65, 513, 777, 1100, 2500, 4096, 4097])
def test_norm_backward_in_place(C, t):
    """dx over dx_add: lanes that share channels (rows that are not whole
    pieces), also of different waves, add the gradient once."""
    say("norm in place", C, t)
    x, dout, gain, add = rnd(1, 700, C, dtype=t), rnd(2, 700, C), rnd(3, C), rnd(4, 700, C, dtype=t)
    _, mean, rstd = srnl.layer_norm_fwd(x, gain, None, stats=True)
    want = srnl.layer_norm_bwd(dout, x, gain, mean, rstd, dx_add=add)
    here = add.clone()
    got = srnl.layer_norm_bwd(dout, x, gain, mean, rstd, dx_add=here, dx=here)
    assert got[0] is here and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("M,K,N", [(3, 40, 24), (100, 333, 517), (700, 72, 523), (5200, 64, 1000), (8200, 264, 2056),
                                   (40, 2000, 64), (70000, 64, 40)])
def test_linear_in_place(M, K, N, t):
    """out over the residual, dx over dx_add: few rows, every tile, a split
    input gradient and the narrow form."""
    say("linear in place", M, K, N, t)
    x, w, r = rnd(1, M, K, dtype=t), rnd(2, N, K, dtype=t), rnd(3, M, N, dtype=t)
    want = srnl.linear_fwd(x, w, act="silu", residual=r)
    here = r.clone()
    assert srnl.linear_fwd(x, w, act="silu", residual=here, out=here) is here
    assert torch.equal(here, want)
    add = rnd(4, M, K, dtype=t)
    want = srnl.linear_bwd(r, x, w, dx_add=add)
    dw, db = abi_linear_bwd(r, x, w, add, add)
    assert all(torch.equal(a, b) for a, b in zip((add, dw, db), want))


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("B,H,W,C", [(3, 9, 7, 64), (2, 5, 6, 33), (90, 57, 7, 16)])
def test_dwconv_in_place(B, H, W, C, t):
    """out over either addend, du over du_add."""
    say("dwconv in place", B, H, W, C, t)
    u, w, a, b = rnd(1, B, H, W, C, dtype=t), rnd(2, C, 3, 3), rnd(3, B, H, W, C, dtype=t), rnd(4, B, H, W, C)
    want = srnl.dwconv_fwd(u, w, None, a, b)
    here = a.clone()
    assert srnl.dwconv_fwd(u, w, None, here, b, out=here) is here and torch.equal(here, want)
    want = srnl.dwconv_fwd(u, w, None, b, a)
    here = a.clone()
    assert torch.equal(srnl.dwconv_fwd(u, w, None, b, here, out=here), want)
    want = srnl.dwconv_bwd(b, u, w, du_add=a)
    L, here = srnl.lib(), a.clone()
    dw, db = torch.empty_like(w), torch.empty(C, device=DEV)
    ws = torch.empty(L.srnl_dwconv_bwd_workspace_bytes(B, H, W, C), dtype=torch.uint8, device=DEV)
    assert L.srnl_dwconv_bwd(b.data_ptr(), 0, u.data_ptr(), B, H, W, C, srnl._dtype_code(u), w.data_ptr(),
                             here.data_ptr(), here.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(),
                             ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert all(torch.equal(p, q) for p, q in zip((here, dw, db), want))


def test_streams_of_another_device_are_refused():
    class Other:                       # what the binding reads of a torch stream
        cuda_stream, device_index = 0, 5

    x, w, g = rnd(1, 4, 8), rnd(2, 16, 8), rnd(3, 8)
    u, cw = rnd(4, 1, 2, 2, 8), rnd(5, 8, 3, 3)
    s = torch.zeros(4, device=DEV)
    for call in (lambda **k: srnl.layer_norm_fwd(x, g, g, **k), lambda **k: srnl.layer_norm_bwd(x, x, g, s, s, **k),
                 lambda **k: srnl.linear_fwd(x, w, **k), lambda **k: srnl.linear_bwd(rnd(6, 4, 16), x, w, **k),
                 lambda **k: srnl.dwconv_fwd(u, cw, **k), lambda **k: srnl.dwconv_bwd(u, u, cw, **k)):
        with pytest.raises(ValueError, match="stream of cuda:5"):
            call(stream=Other)
        call(stream=torch.cuda.current_stream())
