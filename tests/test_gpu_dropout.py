"""Dropout against the generator written out in numpy (Salmon et al., SC'11:
Philox4x32-10), element by element.

Bounds: the scale and the product round once each and the residual's sum once
(u = 2^-24 each, of their values), the output once more (bf16 2^-8, fp32 2^-24
of its value).
"""
import numpy as np
import pytest
import torch

from self_referential_memory_amd import srnl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def philox_bits(count, seed, offset):
    """The 16 bits of elements 0 .. count - 1."""
    m = np.uint64(0xFFFFFFFF)
    blk = np.arange((count + 7) // 8, dtype=np.uint64)
    c = [blk & m, blk >> np.uint64(32), np.full_like(blk, offset & 0xFFFFFFFF), np.full_like(blk, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & m, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, 1).astype(np.uint32)
    return np.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:count]


def test_generator_known_answer():
    """Philox4x32-10's published known answer for counter and key 0: 6627e8d5
    e169c58d bc57ac4c 9b00dbd8."""
    bits = philox_bits(8, 0, 0)
    words = [int(bits[2 * i]) | int(bits[2 * i + 1]) << 16 for i in range(4)]
    assert words == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def rnd(seed, *shape, dtype=F32):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(DEV).to(dtype)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 2048, 2049, 100003])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.99999, 1e-9])
@pytest.mark.parametrize("x_t,r_t,y_t", [(F32, F32, F32), (BF16, BF16, BF16), (F32, None, BF16), (BF16, F32, F32)])
def test_forward_and_backward(n, p, x_t, r_t, y_t):
    print("[dropout]", n, p, x_t, r_t, y_t, flush=True)
    seed, offset = 0xDEADBEEF12345678, (5 << 40) + 17
    x, dout = rnd(n, n, dtype=x_t), rnd(n + 1, n, dtype=y_t)
    res = None if r_t is None else rnd(n + 2, n, dtype=r_t)
    cut = min(int(p * 65536 + 0.5), 65535)
    keep = torch.from_numpy(philox_bits(n, seed, offset).astype(np.int64) >= cut).to(DEV)
    up = 65536 / (65536 - cut)
    y = srnl.dropout_fwd(x, p, seed, offset, residual=res, out_dtype=y_t)
    part = torch.where(keep, x.double() * up, 0.0)
    ref = part + (0 if res is None else res.double())
    bound = 2 * U * part.abs() + U * ref.abs()
    assert y.dtype == y_t and bool(((y.double() - ref).abs() <= bound + HALF[y_t] * ref.abs()).all())
    if res is not None:
        assert torch.equal(y[~keep], res.float().to(y_t)[~keep])
    dx = srnl.dropout_bwd(dout, p, seed, offset, dtype=x_t)
    ref = torch.where(keep, dout.double() * up, 0.0)
    assert dx.dtype == x_t and bool(((dx.double() - ref).abs() <= (2 * U + HALF[x_t]) * ref.abs()).all())
    add = rnd(n + 3, n, dtype=x_t)
    dx = srnl.dropout_bwd(dout, p, seed, offset, dtype=x_t, dx_add=add)
    s = ref + add.double()
    assert bool(((dx.double() - s).abs() <= 2 * U * ref.abs() + (U + HALF[x_t]) * s.abs()).all())


def test_what_is_dropped_may_be_anything():
    n = 4096
    keep = torch.from_numpy(philox_bits(n, 3, 0).astype(np.int64) >= 32768).to(DEV)
    x = torch.where(keep, rnd(1, n), torch.tensor(float("nan"), device=DEV))
    x[::2] = torch.where(keep[::2], x[::2], torch.tensor(float("inf"), device=DEV))
    y = srnl.dropout_fwd(x, 0.5, 3)
    assert y.isfinite().all() and not y[~keep].any() and torch.equal(y[keep], 2 * x[keep])


def test_counter_draws_new_masks_in_a_captured_graph():
    x, counter = rnd(1, 5000), torch.zeros(1, dtype=torch.int64, device=DEV)
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        srnl.dropout_fwd(x, 0.3, 11, 100, counter=counter, out=y)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        counter += 1
        srnl.dropout_fwd(x, 0.3, 11, 100, counter=counter, out=y)
    for step in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, srnl.dropout_fwd(x, 0.3, 11, 100 + step))
        assert not torch.equal(y, srnl.dropout_fwd(x, 0.3, 11, 100))


def test_autograd_keeps_seed_offset_and_counter():
    x, res = rnd(1, 30, 77).requires_grad_(), rnd(2, 30, 77, dtype=BF16).requires_grad_()
    w = rnd(3, 30, 77)
    counter = torch.full((1,), 9, dtype=torch.int64, device=DEV)
    y = srnl.dropout(x, 0.4, 5, 6, residual=res, counter=counter)
    counter += 1                          # the next step's, before this one's backward
    dx, dr = torch.autograd.grad((y * w).sum(), (x, res))
    assert torch.equal(y, srnl.dropout_fwd(x.detach(), 0.4, 5, 15, residual=res.detach()))
    assert torch.equal(dx, srnl.dropout_bwd(w, 0.4, 5, 15)) and torch.equal(dr, w.to(BF16))


def test_shapes_and_negative_offsets_count_modulo_2_64():
    x = rnd(1, 3, 5, 7)
    assert torch.equal(srnl.dropout_fwd(x, 0.5, -1, -2), srnl.dropout_fwd(x, 0.5, 2 ** 64 - 1, 2 ** 64 - 2))
    assert torch.equal(srnl.dropout_fwd(x, 0.5, 1).flatten(), srnl.dropout_fwd(x.flatten(), 0.5, 1))
    assert srnl.dropout_fwd(x[:0], 0.5, 1).shape == (0, 5, 7)
