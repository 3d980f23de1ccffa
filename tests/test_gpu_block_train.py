"""The layers as a user runs them together: the differentiable residual block
(srnl.block) and the layers' autograd nodes, against the block written in
float64 (oracle/srnl_grad.py's operator and elementary torch operations on the
CPU, differentiated by autograd), on side streams and in captured graphs.

Bars: the operator's (1e-4 forward, 1e-3 gradients, relative to the largest
magnitude), as in the operator's own gradient tests; a bf16 output or
gradient may be half a step (2^-8 of each element) further off.
"""
import numpy as np
import pytest
import torch

from oracle import srnl_grad
from self_referential_memory_amd import srnl, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def block64(x, st, sc, bw, heads, d, mask, ln_eps, **kw):
    def norm(v, g, b):
        m = v.mean(-1, keepdim=True)
        return (v - m) / ((v - m).square().mean(-1, keepdim=True) + ln_eps).sqrt() * g + b

    H, W = x.shape[1:3]
    u = norm(x, bw["ln1_w"], bw["ln1_b"])
    q = u @ bw["wq"].t()
    _, s = srnl_grad.forward(u, st, sc, heads, d, mask, q, **kw)
    p = torch.nn.functional.pad(u, (0, 0, 1, 1, 1, 1))
    conv = sum(p[:, a:a + H, e:e + W] * bw["dw_w"][:, a, e] for a in range(3) for e in range(3))
    h = x + conv + bw["dw_b"] + s
    v = norm(h, bw["ln2_w"], bw["ln2_b"])
    z = v @ bw["w1"].t() + bw["b1"]
    return h + (z * torch.special.erfc(-z / 2 ** 0.5) / 2) @ bw["w2"].t() + bw["b2"]


def setup(wl, F, wdt=BF16):
    bw = synth.block_weights(wl.seed, wl.C, F)
    dt = BF16 if wl.dtype == "bf16" else F32
    leaf = lambda a, t=F32: torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(t).requires_grad_()
    x, st, sc = leaf(wl.x, dt), leaf(wl.states), leaf(wl.scales)
    w = {k: leaf(getattr(bw, k), wdt if k in ("wq", "w1", "w2") else F32) for k in srnl.BLOCK_KEYS}
    return x, st, sc, w


def near(got, ref, bar, what):
    ref = ref.detach()
    step = 2.0 ** -8 * ref.abs() if got.dtype == BF16 else 0.0
    over = (got.detach().double().cpu() - ref).abs() - bar * ref.abs().max() - step
    assert bool((over <= 0).all()), f"{what}: over by {over.max().item():.2e}"


@pytest.mark.parametrize("B,H,W,heads,d,F,dtype,wdt,mask", [
    (2, 5, 7, 2, 32, 256, "f32", BF16, 15), (1, 4, 6, 1, 16, 40, "f32", F32, 15),
    (2, 6, 5, 4, 32, 512, "bf16", BF16, 15), (1, 3, 9, 3, 8, 96, "bf16", F32, 5),
    (1, 7, 7, 3, 64, 768, "f32", BF16, 15)])
def test_block_forward_and_gradients(B, H, W, heads, d, F, dtype, wdt, mask):
    print("[block]", B, H, W, heads, d, F, dtype, wdt, mask, flush=True)
    wl = synth.make("blk_train", B, H, W, heads * d, heads, d, dtype, 41, state_std=0.5)
    x, st, sc, w = setup(wl, F, wdt)
    out = srnl.block(x, st, sc, w, heads, d, mask, 1e-5)
    g = torch.randn(out.shape, generator=torch.Generator().manual_seed(1)).to(DEV).to(out.dtype)
    out.backward(g)
    c = {k: v.detach().double().cpu().requires_grad_() for k, v in
         dict(x=x, st=st, sc=sc, **w).items()}
    ref = block64(c["x"], c["st"], c["sc"], c, heads, d, mask, 1e-5, alpha_max=0.9, eps=1e-6)
    ref.backward(g.double().cpu())
    near(out, ref, 1e-4, "out")
    for k, t in dict(x=x, st=st, sc=sc, **w).items():
        near(t.grad, c[k].grad, 1e-3, f"d{k}")
    if wdt == BF16 and wl.C in (32, 64, 128, 192, 256, 512):      # the fused inference block
        fused = srnl.block_fwd(x.detach(), st.detach(), srnl.block_weights(
            {k: v.detach() for k, v in w.items()}, sc.detach()), heads, d, mask)
        near(fused, out.detach().double().cpu(), 1e-4 if dtype == "f32" else 2.0 ** -8, "block_fwd")


def test_block_gradient_against_differences():
    """Directional derivatives of a fp32 block against central differences of
    the float64 block: along random directions of every input together."""
    wl = synth.make("blk_fd", 1, 4, 5, 32, 1, 32, "f32", 42, state_std=0.5)
    x, st, sc, w = setup(wl, 64, F32)
    named = dict(x=x, st=st, sc=sc, **w)
    g = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(DEV)
    srnl.block(x, st, sc, w, 1, 32).backward(g)
    gen = torch.Generator().manual_seed(3)
    base = {k: v.detach().double().cpu() for k, v in named.items()}
    for _ in range(3):
        dirs = {k: torch.randn(v.shape, generator=gen, dtype=torch.float64) * 0.1 for k, v in base.items()}
        f = []
        for s in (1e-4, -1e-4):
            c = {k: v + s * dirs[k] for k, v in base.items()}
            f.append((block64(c["x"], c["st"], c["sc"], c, 1, 32, 15, 1e-5, alpha_max=0.9, eps=1e-6)
                      * g.double().cpu()).sum())
        fd = (f[0] - f[1]) / 2e-4
        an = sum((named[k].grad.double().cpu() * dirs[k]).sum() for k in base)
        size = sum((named[k].grad.double().cpu() * dirs[k]).abs().sum() for k in base)
        assert abs(an - fd) <= 1e-4 * size


def test_layers_as_autograd_nodes():
    """The nodes' gradients are the backward entry points', for inputs that
    come in and gradients that go out in either type, broadcast and strided
    gradients included; without any gradient wanted nothing is kept."""
    x = torch.randn(3, 20, 64, device=DEV).to(BF16).requires_grad_()
    gain, bias = (torch.randn(64, device=DEV).requires_grad_() for _ in range(2))
    w = torch.randn(96, 64, device=DEV).to(BF16).requires_grad_()
    b = torch.randn(96, device=DEV).requires_grad_()
    r = torch.randn(3, 20, 96, device=DEV).requires_grad_()
    n = srnl.layer_norm(x, gain, bias, out_dtype=F32)
    y = srnl.linear(n, w, b, act="silu", residual=r, out_dtype=BF16)
    y.sum().backward()                                        # an expanded gradient
    dy = torch.ones_like(y)
    n0, mean, rstd = srnl.layer_norm_fwd(x.detach(), gain, bias, out_dtype=F32, stats=True)
    pre = srnl.linear_fwd(n0, w, b, act="silu", keep_pre=True)[1]
    dn, dw, db = srnl.linear_bwd(dy, n0, w.detach(), pre, act="silu")
    dx, dg, dbi = srnl.layer_norm_bwd(dn, x.detach(), gain, mean, rstd)
    for got, want in ((x.grad, dx), (gain.grad, dg), (bias.grad, dbi), (w.grad, dw.to(BF16)),
                      (b.grad, db), (r.grad, dy.to(F32))):
        assert got.dtype == want.dtype and torch.equal(got, want)
    u = torch.randn(2, 6, 5, 64, device=DEV, requires_grad=True)
    cw = torch.randn(64, 3, 3, device=DEV, requires_grad=True)
    a1 = torch.randn(2, 6, 5, 64, device=DEV).to(BF16).requires_grad_()
    srnl.dwconv(u, cw, None, a1).transpose(1, 2).float().square().sum().backward()
    y = srnl.dwconv_fwd(u.detach(), cw.detach(), None, a1.detach())
    du, dcw, _ = srnl.dwconv_bwd(2 * y, u.detach(), cw.detach())
    assert torch.equal(u.grad, du) and torch.equal(cw.grad, dcw)
    assert torch.equal(a1.grad, (2 * y).to(BF16))
    with torch.no_grad():
        assert srnl.linear(n0, w, b, act="gelu").grad_fn is None
    only_b = srnl.linear(n0, w.detach(), b)
    b.grad = None
    only_b.sum().backward()
    assert b.grad is not None


def test_gradients_from_any_address():
    """A joined output's gradient comes back in slices that may start at any
    element."""
    x = torch.randn(3, 5, device=DEV, requires_grad=True)
    w = torch.randn(7, 5, device=DEV, requires_grad=True)
    g = torch.randn(7, device=DEV, requires_grad=True)
    u = torch.randn(1, 1, 3, 7, device=DEV, requires_grad=True)
    cw = torch.randn(7, 3, 3, device=DEV, requires_grad=True)
    leaves = (x, w, g, u, cw)
    seed = torch.randn(10, 7, device=DEV)
    parts = [torch.zeros(1, 7, device=DEV), srnl.linear(x, w), srnl.layer_norm(x @ w.t(), g, None),
             srnl.dwconv(u, cw).view(3, 7)]
    got = torch.autograd.grad(torch.cat(parts), leaves, seed)
    want = [torch.zeros_like(t) for t in leaves]
    for p, a, b in ((parts[1], 1, 4), (parts[2], 4, 7), (parts[3], 7, 10)):
        p = srnl.linear(x, w) if a == 1 else srnl.layer_norm(x @ w.t(), g, None) if a == 4 \
            else srnl.dwconv(u, cw).view(3, 7)
        for t, v in zip(want, torch.autograd.grad(p, leaves, seed[a:b].clone(), allow_unused=True)):
            if v is not None:
                t += v
    # the same terms (below 100) in another order: three additions, each off by
    # 2^-24 of a sum below 200
    for a, b in zip(got, want):
        assert (a - b).abs().max() <= 3 * 200 * 2.0 ** -24


def test_layers_on_a_side_stream():
    """Inputs made on the current stream, calls on another one that waits for
    it: the workspaces the binding frees on return are not handed out again
    before that stream is done."""
    x = torch.randn(40000, 64, device=DEV)
    w = torch.randn(256, 64, device=DEV).to(BF16)
    dout = torch.randn(40000, 256, device=DEV)
    gain = torch.ones(64, device=DEV)
    want = srnl.linear_bwd(dout, x, w)
    y, m, r = srnl.layer_norm_fwd(x, gain, None, stats=True)
    wantn = srnl.layer_norm_bwd(y, x, gain, m, r)
    g4 = x.view(4, 100, 100, 64)
    cw = torch.randn(64, 3, 3, device=DEV)
    wantc = srnl.dwconv_bwd(g4, g4, cw)
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        got = srnl.linear_bwd(dout, x, w, stream=side)
        gotn = srnl.layer_norm_bwd(y, x, gain, m, r, stream=side)
        gotc = srnl.dwconv_bwd(g4, g4, cw, stream=side)
        junk = [torch.full((1 << 22,), 3.0, device=DEV) for _ in range(6)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip((*got, *gotn, *gotc), (*want, *wantn, *wantc)):
            assert torch.equal(a, b)
        del junk


def test_layers_in_captured_graphs():
    """Two graphs captured over one memory pool, replayed in turn with eager
    work between: every replay gives the eager results for the inputs that
    are there."""
    x = torch.randn(3000, 128, device=DEV)
    w1, w2 = torch.randn(200, 128, device=DEV).to(BF16), torch.randn(128, 200, device=DEV).to(BF16)
    gain, bias = torch.randn(128, device=DEV), torch.randn(128, device=DEV)
    u = torch.randn(2, 30, 50, 128, device=DEV)
    cw, cb = torch.randn(128, 3, 3, device=DEV), torch.randn(128, device=DEV)

    def mlp():
        n, m, r = srnl.layer_norm_fwd(x, gain, bias, stats=True)
        a, z = srnl.linear_fwd(n, w1, act="gelu", keep_pre=True)
        y = srnl.linear_fwd(a, w2, bias, residual=x)
        da, dw2, db2 = srnl.linear_bwd(y, a, w2)
        dn, dw1, _ = srnl.linear_bwd(da, n, w1, z, act="gelu", need_db=False)
        return (y, dw1, dw2, db2, *srnl.layer_norm_bwd(dn, x, gain, m, r, dx_add=y))

    def conv():
        y = srnl.dwconv_fwd(u, cw, cb)
        return (y, *srnl.dwconv_bwd(y, u, cw))

    graphs = []
    pool = None
    for f in (mlp, conv):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = f()
        pool = g.pool()
        graphs.append((f, g, out))
    for k in range(4):
        x.normal_()
        u.normal_()
        want = [[t.clone() for t in f()] for f, _, _ in graphs]
        for (f, g, out), w in zip(graphs, want):
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, w):
                assert torch.equal(a, b), k
