"""The gated delta rule where it can go wrong: gates of 0 and -infinity, tokens
past the end, slices, states taken up and handed on, streams, graphs, offsets
past 32 bits, gradients against differences. Bounds as in test_gpu_gated_delta."""
import pytest
import torch

from self_referential_memory_amd import srnl
from tests import delta_oracle
from tests.test_gpu_gated_delta import BF16, DEV, F32, chunk_tol, close, on_gpu, say, step_tol

pytestmark = pytest.mark.gpu


def call(x, **kw):
    return srnl.gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"], lengths=x["lengths"],
                                norm_eps=1e-6, **kw)


def back(x, dout, rec, dstate=None, **kw):
    return srnl.gated_delta_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], rec, state=x["state"], dstate=dstate,
                                lengths=x["lengths"], norm_eps=1e-6, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_at_their_ends(dtype):
    """exp(-inf) = 0 starts the state anew, beta = 0 writes nothing, g = 0 keeps
    everything, g = -500 leaves nothing and no NaN."""
    d = delta_oracle.inputs(1, 2, 150, 2, 2, 32, 24, dtype, state=True)
    d["g"][:, 40] = float("-inf")
    d["g"][:, 64:66] = float("-inf")
    d["g"][0, 100:120] = -500.0
    d["g"][1, 70:] = 0.0
    d["beta"][:, 30:50] = 0.0
    d["beta"][:, 90] = 1.0
    dout = torch.randn(2, 150, 2, 24, generator=torch.Generator().manual_seed(2)).to(dtype)
    # the reference's gradient of exp at -inf is 0 x anything: it is given there
    safe = dict(d, g=d["g"].clamp(min=-2000.0))
    ref, S, terms, grads = delta_oracle.reference(safe, norm_eps=1e-6, dout=dout)
    x = on_gpu(d)
    out, S1, rec = call(x, record=True)
    tol = chunk_tol(150, 32, dtype)
    close(out, ref, tol, "out", 2, terms)
    close(S1, S, tol, "state", 1)
    got = back(x, dout.to(DEV), rec)
    for name, t in zip(("q", "k", "v", "g", "beta", "state"), got):
        close(t, grads[name], 3 * tol, "d" + name, 1 if name == "state" else 2)
    # d exp(g) is 0 there: what is left is the rounding of sums over the chunk's other
    # pairs, which enter by row and leave by column: at most 2 x 64 additions, u each,
    # of sums no larger than 64 times the largest gradient of a gate
    assert got[3][:, 40].abs().max() <= 2 * 64 * 64 * 2.0 ** -24 * got[3].abs().max()
    st = x["state"].clone()
    o, S2 = srnl.gated_delta_step(x["q"][:, 40:41].contiguous(), x["k"][:, 40:41].contiguous(),
                                  x["v"][:, 40:41].contiguous(), x["g"][:, 40:41].contiguous(),
                                  x["beta"][:, 40:41].contiguous(), st, norm_eps=1e-6)
    assert not S2.any() and not o.any()               # beta is 0 there too


def test_what_lies_past_the_end_is_not_read():
    d = delta_oracle.inputs(3, 4, 140, 1, 2, 40, 48, BF16, state=True, lengths=(0, 1, 70, 128))
    x = on_gpu(d)
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    dout = torch.randn(4, 140, 2, 48, device=DEV).bfloat16()
    bad = dout.clone()
    for b, n in enumerate((0, 1, 70, 128)):
        for name in ("q", "k", "v", "g", "beta"):
            y[name][b, n:] = float("nan")
        bad[b, n:] = float("inf")
    o1, s1, r1 = call(x, record=True)
    o2, s2, r2 = call(y, record=True)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)
    for a, b in zip(back(x, dout, r1), back(y, bad, r2)):
        assert torch.equal(a, b)
    for t in (1, 3):
        z, w = ({n: (v[:, :t].contiguous() if n in ("q", "k", "v", "g", "beta") else v) for n, v in u.items()} for u in (x, y))
        a, b = (srnl.gated_delta_step(u["q"], u["k"], u["v"], u["g"], u["beta"], x["state"].clone(), lengths=x["lengths"])
                for u in (z, w))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slices_of_one_projection(dtype):
    B, T, Hk, H, Dk, Dv = 2, 100, 2, 4, 24, 40
    d = on_gpu(delta_oracle.inputs(4, B, T, Hk, H, Dk, Dv, dtype, state=True))
    width = 2 * Hk * Dk + H * Dv + 16
    p = torch.full((B, T, width), float("nan"), device=DEV, dtype=dtype)
    cut, x = 0, dict(d)
    for n, h, w in (("v", H, Dv), ("q", Hk, Dk), ("k", Hk, Dk)):
        p[..., cut:cut + h * w] = d[n].flatten(2)
        x[n] = p[..., cut:cut + h * w].unflatten(2, (h, w))
        cut += h * w
    dout = torch.randn(B, T, H, Dv, device=DEV).to(dtype)
    o1, s1, r1 = call(d, record=True)
    o2, s2, r2 = call(x, record=True)
    assert torch.equal(o1, o2) and torch.equal(s1, s2) and torch.equal(r1, r2)
    for a, b in zip(back(d, dout, r1), back(x, dout, r2)):
        assert torch.equal(a, b)
    one, two = ({n: (t[:, :2] if n in ("q", "k", "v") else t[:, :2].contiguous() if n in ("g", "beta") else t)
                 for n, t in u.items()} for u in (d, x))
    one = {n: t.contiguous() if n in ("q", "k", "v") else t for n, t in one.items()}
    with pytest.raises(ValueError, match="contiguous"):       # two of a hundred tokens: items do not follow on
        srnl.gated_delta_step(two["q"], one["k"], one["v"], one["g"], one["beta"], d["state"].clone())
    a = srnl.gated_delta_step(*(one[n][:1] for n in ("q", "k", "v", "g", "beta")), d["state"][:1].clone())
    b = srnl.gated_delta_step(*(two[n][:1] for n in ("q", "k", "v", "g", "beta")), d["state"][:1].clone())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cut", [1, 63, 64, 100])
def test_states_handed_on(dtype, cut):
    """A sequence in two calls, and its tail token by token."""
    d = delta_oracle.inputs(5, 2, 130, 1, 2, 64, 32, dtype, state=True)
    ref, S, terms = delta_oracle.reference(d, norm_eps=1e-6)
    x = on_gpu(d)
    tol = 2 * chunk_tol(130, 64, dtype)

    def part(lo, hi, state):
        return {n: t[:, lo:hi].contiguous() if n in ("q", "k", "v", "g", "beta") else t
                for n, t in x.items()} | {"state": state}

    kept = x["state"].clone()
    o1, s1 = call(part(0, cut, kept), state_out=kept)          # in place
    assert s1 is kept
    o2, s2 = call(part(cut, 130, s1))
    close(torch.cat((o1, o2), 1), ref, tol, "out", 2, terms)
    close(s2, S, tol, "state", 1)
    outs, st = [o1], s1.clone()
    for lo in range(cut, 130, 7):
        y = part(lo, min(lo + 7, 130), None)
        o, st = srnl.gated_delta_step(y["q"], y["k"], y["v"], y["g"], y["beta"], st, norm_eps=1e-6)
        outs.append(o)
    close(torch.cat(outs, 1), ref, tol + step_tol(130, 64), "out", 2, terms)
    close(st, S, tol + step_tol(130, 64), "state", 1)


def test_no_tokens_and_no_items():
    for B, T in ((2, 0), (0, 5)):
        x = on_gpu(delta_oracle.inputs(6, B, T, 1, 2, 16, 24, BF16, state=True))
        out, s, rec = call(x, record=True)
        assert out.shape == (B, T, 2, 24) and torch.equal(s, x["state"])
        dst = torch.randn_like(s)
        got = back(x, torch.empty_like(out), rec, dst)
        assert got[0].shape == x["q"].shape and got[3].shape == x["g"].shape and torch.equal(got[5], dst)
        o, s = srnl.gated_delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"].clone())
        assert o.shape == out.shape and torch.equal(s, x["state"])


def test_scale_zero_keys_and_strong_writes():
    """A key of zeros has no direction; beta up to 2 reflects; any scale."""
    d = delta_oracle.inputs(7, 1, 100, 2, 2, 48, 16, F32)
    d["k"][0, 10:20] = 0.0
    d["q"][0, 30] = 0.0
    d["beta"] *= 2.0
    dout = torch.randn(1, 100, 2, 16, generator=torch.Generator().manual_seed(8))
    ref, S, terms, grads = delta_oracle.reference(d, scale=-0.7, norm_eps=1e-4, dout=dout)
    x = on_gpu(d)
    kw = dict(scale=-0.7, norm_eps=1e-4)
    args = tuple(x[n] for n in ("q", "k", "v", "g", "beta"))
    out, S1, rec = srnl.gated_delta_fwd(*args, record=True, **kw)
    tol = 2 * chunk_tol(100, 48, F32)
    close(out, ref, tol, "out", 2, terms)
    close(S1, S, tol, "state", 1)
    for name, t in zip(("q", "k", "v", "g", "beta"), srnl.gated_delta_bwd(dout.to(DEV), *args, rec, **kw)):
        close(t, grads[name], 6 * tol, "d" + name, 2)


def test_gradients_against_differences():
    d = delta_oracle.inputs(9, 1, 70, 1, 2, 16, 8, F32, state=True)
    gen = torch.Generator().manual_seed(10)
    w, ws = torch.randn(1, 70, 2, 8, generator=gen).double(), torch.randn(1, 2, 16, 8, generator=gen).double()
    x = {n: None if t is None else t.to(DEV).requires_grad_(t.is_floating_point()) for n, t in d.items()}
    out, S = srnl.gated_delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"], norm_eps=1e-6)
    names = ("q", "k", "v", "g", "beta", "state")
    grads = torch.autograd.grad((out.double() * w.to(DEV)).sum() + (S.double() * ws.to(DEV)).sum(), [x[n] for n in names])

    def loss(**change):
        y = {n: d[n].double() + change.get(n, 0.0) for n in names}
        o, s, _ = delta_oracle.rule(y["q"], y["k"], y["v"], y["g"], y["beta"], y["state"], None, None, 1e-6)
        return ((o * w).sum() + (s * ws).sum()).item()

    for n, t in zip(names, grads):
        v = torch.randn(d[n].shape, generator=gen).double()
        h = 1e-5
        num = (loss(**{n: h * v}) - loss(**{n: -h * v})) / (2 * h)
        ana = (t.cpu().double() * v).sum().item()
        # the difference's h^2, and the gradient's bound as a whole
        bound = (3 * chunk_tol(70, 16, F32) + 1e-6) * (t.cpu().double().norm() * v.norm()).item()
        assert abs(num - ana) <= bound, (n, num, ana)


def test_autograd_wants_and_misses_outputs():
    x = on_gpu(delta_oracle.inputs(12, 2, 66, 1, 2, 24, 16, BF16, state=True))
    leaves = {n: x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta", "state")}
    args = tuple(leaves[n] for n in ("q", "k", "v", "g", "beta", "state"))
    out, S = srnl.gated_delta(*args, norm_eps=1e-6)
    o2, s2, rec = call(x, record=True)
    assert torch.equal(out, o2) and torch.equal(S, s2)
    w = torch.randn_like(S)
    zero = torch.zeros_like(out)
    for a, b in zip(torch.autograd.grad((S * w).sum(), args, retain_graph=True), back(x, zero, rec, w)):
        assert torch.equal(a, b)                      # the output unused
    v = torch.randn_like(out)
    for a, b in zip(torch.autograd.grad((out * v).sum(), args), back(x, v, rec)):
        assert torch.equal(a, b)                      # the states unused
    with torch.no_grad():
        assert srnl.gated_delta(*args, norm_eps=1e-6)[0].grad_fn is None


def test_other_streams_and_two_calls_at_once():
    xs = [on_gpu(delta_oracle.inputs(20 + i, 4, 300, 2, 2, 64, 64, BF16, state=True)) for i in range(2)]
    douts = [torch.randn(4, 300, 2, 64, device=DEV).bfloat16() for _ in xs]
    want = []
    for x, d in zip(xs, douts):
        o, s, r = call(x, record=True)
        want.append((o, s, *back(x, d, r)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []                               # kept: their memory is in use on the streams
    for _ in range(3):
        for x, d, st in zip(xs, douts, streams):
            o, s, r = call(x, record=True, stream=st)
            with torch.cuda.stream(st):
                got.append((o, s, r, *back(x, d, r)))
    torch.cuda.synchronize()
    for i, b in enumerate(got):
        a = want[i % 2]
        assert all(torch.equal(p, q) for p, q in zip(a, b[:2] + b[3:]))


def test_captured_and_replayed():
    """A training step and a serving step in one graph each, replayed on new
    inputs with eager calls between."""
    x = on_gpu(delta_oracle.inputs(30, 2, 100, 1, 2, 32, 48, BF16, state=True))
    dout = torch.randn(2, 100, 2, 48, device=DEV).bfloat16()
    one = {n: t[:, :1].contiguous() if n in ("q", "k", "v", "g", "beta") else t for n, t in x.items()}
    st = x["state"].clone()
    side = torch.cuda.Stream()

    def train():
        o, s, r = call(x, record=True)
        return (o, s, *back(x, dout, r))

    def serve():
        return srnl.gated_delta_step(one["q"], one["k"], one["v"], one["g"], one["beta"], st, norm_eps=1e-6)

    with torch.cuda.stream(side):
        train(), serve()
    side.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        res = train()
    with torch.cuda.graph(g2):
        tok = serve()
    for seed in range(40, 44):
        new = on_gpu(delta_oracle.inputs(seed, 2, 100, 1, 2, 32, 48, BF16, state=True))
        for n in ("q", "k", "v", "g", "beta", "state"):
            x[n].copy_(new[n])
            if n != "state":
                one[n].copy_(new[n][:, :1])
        st.copy_(new["state"])
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        want = train()
        assert all(torch.equal(a, b) for a, b in zip(res, want))
        fresh = new["state"].clone()
        o, s = srnl.gated_delta_step(one["q"], one["k"], one["v"], one["g"], one["beta"], fresh, norm_eps=1e-6)
        assert torch.equal(tok[0], o) and torch.equal(st, s)


def test_offsets_past_32_bits():
    """Tokens 65536 elements apart, 40000 of them: 2.6e9 elements between the
    first and the last; states of 9300 sequences x 16 heads."""
    T, width = 40000, 65536
    p = torch.empty(1, T, width, device=DEV, dtype=BF16)
    d = on_gpu(delta_oracle.inputs(50, 1, T, 1, 1, 16, 16, BF16))
    x = dict(d)
    for i, n in enumerate(("q", "k", "v")):
        cut = (0, 32768, width - 16)[i]
        p[..., cut:cut + 16] = d[n].flatten(2)
        x[n] = p[..., cut:cut + 16].unflatten(2, (1, 16))
    dout = torch.randn(1, T, 1, 16, device=DEV).bfloat16()
    o1, s1, r1 = call(d, record=True)
    o2, s2, r2 = call(x, record=True)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)
    for a, b in zip(back(d, dout, r1)[:5], back(x, dout, r2)[:5]):
        assert torch.equal(a, b)
    del p, x, r1, r2
    B, H = 9300, 16
    say("states", B * H * 128 * 128 * 4 / 2 ** 30, "GiB")
    small = on_gpu(delta_oracle.inputs(51, 2, 1, 16, 16, 128, 128, BF16, state=True))
    st = torch.zeros(B, H, 128, 128, device=DEV)
    st[-2:] = small["state"]
    big = {n: torch.zeros((B,) + small[n].shape[1:], device=DEV, dtype=small[n].dtype) for n in ("q", "k", "v", "g", "beta")}
    for n in big:
        big[n][-2:] = small[n]
    o, _ = srnl.gated_delta_step(big["q"], big["k"], big["v"], big["g"], big["beta"], st, norm_eps=1e-6)
    # the same width of block for both: 32 sequences and more take the wider one
    pad = {n: torch.cat([small[n]] * 16) for n in big}
    o1, s1 = srnl.gated_delta_step(pad["q"], pad["k"], pad["v"], pad["g"], pad["beta"], torch.cat([small["state"]] * 16),
                                   norm_eps=1e-6)
    assert torch.equal(o[-2:], o1[-2:]) and torch.equal(st[-2:], s1[-2:])
    assert not st[:-2].any()


@pytest.mark.parametrize("Dv", [16, 40])
def test_a_large_call_as_its_parts(Dv):
    """More chunks than the caches hold, and more blocks than compute units, are stored
    and cut in their own ways: the same values, bit for bit, as two calls of half of it."""
    B, T, H = 200, 900, 1
    assert B * H * 15 * 2 * 64 * 64 * 6 > 128 << 20 > B // 2 * H * 15 * 2 * 64 * 64 * 6
    g = torch.Generator(DEV).manual_seed(Dv)
    lengths = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int()
    q, k, v, dout = (torch.randn(B, T, H, n, generator=g, device=DEV).bfloat16() for n in (16, 16, Dv, Dv))
    gate, beta = -torch.rand(B, T, H, generator=g, device=DEV), torch.rand(B, T, H, generator=g, device=DEV)
    dstate = torch.randn(B, H, 16, Dv, generator=g, device=DEV)

    def both(s):
        part = dict(q=q[s], k=k[s], v=v[s], g=gate[s], beta=beta[s], state=None, lengths=lengths[s])
        out, S, rec = call(part, record=True)
        return [out, S] + [t for t in back(part, dout[s], rec, dstate=dstate[s]) if t is not None]

    whole = both(slice(0, B))
    for s in (slice(0, B // 2), slice(B // 2, B)):
        for a, b in zip(whole, both(s)):
            assert torch.equal(a[s], b)
            assert b.isfinite().all()
