"""Group norm's statistics over long maps that begin with a cell far out: the
variance is about the mean, and no sum cancels, wherever that cell lies.

Bounds, fixed before the first run; u = 2^-24. A thread joins its cells in fours,
then lanes, slabs and the channels of a group (1024 threads and 32 steps) join: at
most `chain` additions of positive terms and as many of their own roundings, so the
variance is off by 2 chain u of itself, rstd by half of that and 4 u. The mean
rounds at each join, by u of the largest slab's mean, and its sums by chain u of the
cells' mean distance. (Squares about a thread's first cell would be off by u times
the cells to the power of 1.5.)
"""
import pytest
import torch

from self_referential_memory_amd import srnl

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def slabs_of(B, S, C):
    """(cells of a slab, lanes that share them)"""
    v = next(n for n in (8, 4, 2, 1) if C % n == 0)
    lanes = max(1, 256 // (C // v))
    items = B * -(-(C // v) // 256)
    n = min(-(-1024 // items), -(-S // (8 * lanes)))
    return -(-S // n), lanes


@pytest.mark.parametrize("far", [1e3, 1e4])
@pytest.mark.parametrize("offset", [0.0, 1000.0])
@pytest.mark.parametrize("B,S,C,G,dtype", [
    (4, 60000, 255, 1, F32), (1, 300000, 255, 5, F32), (32, 7600, 2048, 1, BF16), (1, 40000, 250, 2, F32),
    (2, 20011, 20, 4, BF16)])
def test_first_cell_far_out(B, S, C, G, dtype, offset, far):
    print("[gnorm outliers]", B, S, C, G, dtype, offset, far, flush=True)
    gen = torch.Generator("cuda:0").manual_seed(S)
    x = torch.randn(B, S, C, generator=gen, device="cuda:0") + offset
    rows, lanes = slabs_of(B, S, C)
    x[:, 0, ::C // G] += far                # a thread's first cell
    x = x.to(dtype)
    y, mean, rstd = srnl.group_norm_fwd(x, G, None, None, 1e-5, stats=True)
    chain = rows / lanes / 4 + lanes + -(-S // rows) * (C // G) / 1024 + 32
    for b in range(B):
        for g in range(G):
            X = x[b, :, g * (C // G):(g + 1) * (C // G)].double()
            m = X.mean()
            d = (X - m).abs()
            r = (d.square().mean() + 1e-5).rsqrt()
            slab = X[::rows].abs().max().item()
            assert abs(mean[b, g].item() - m.item()) <= chain * U * d.mean().item() + 4 * U * slab, "mean"
            assert abs(rstd[b, g].item() / r.item() - 1) <= (chain + 4) * U, "rstd"
    assert y.isfinite().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slabs_of_constant_offset_and_infinite_items(dtype):
    """What holds for a slice holds for a map cut into slabs: a constant group's
    variance is 0, an offset keeps its digits, an infinity stays in its group."""
    gen = torch.Generator("cuda:0").manual_seed(5)
    B, S, C, G = 5, 9001, 64, 16                       # 8 slices an item, of more than 14 cells a thread
    x = torch.randn(B, S, C, generator=gen, device="cuda:0")
    gain, bias = (torch.randn(C, generator=gen, device="cuda:0") for _ in range(2))
    x[0] = 7.25
    x[1] += 1e4 if dtype == F32 else 100.0
    x = x.to(dtype)
    x[2, 0, 5] = float("inf")                          # a thread's first cell
    x[3, 8999, 5] = float("-inf")
    x[4, 4500, 9] = float("nan")
    y, mean, rstd = srnl.group_norm_fwd(x, G, gain, bias, stats=True, out_dtype=F32)
    assert torch.equal(y[0], bias.expand(S, C)) and bool((mean[0] == 7.25).all())
    X = x[1].double().reshape(S, G, 4)
    m = X.mean((0, 2), keepdim=True)
    r = (X.sub(m).square().mean((0, 2), keepdim=True) + 1e-5).rsqrt()
    # joins: 8 cells and a batch's steps a thread, 32 lanes, slabs of 4 channels by 1024
    assert ((rstd[1].double() / r[0, :, 0] - 1).abs() <= 100 * U).all()
    assert ((mean[1].double() - m[0, :, 0]).abs() <= 4 * U * m[0, :, 0].abs() + 100 * U).all()
    clean = x.clone()
    for b, s, c, g in ((2, 0, 5, 1), (3, 8999, 5, 1), (4, 4500, 9, 2)):
        clean[b, s, c] = 0.0
        rest = [j for j in range(C) if j // 4 != g]
        assert y[b, :, 4 * g:4 * g + 4].isnan().all() and y[b][:, rest].isfinite().all()
    y2 = srnl.group_norm_fwd(clean, G, gain, bias, out_dtype=F32)
    bad = torch.zeros(B, C, dtype=torch.bool, device="cuda:0")
    bad[2, 4:8], bad[3, 4:8], bad[4, 8:12] = True, True, True
    assert torch.equal(torch.where(bad[:, None], 0.0, y), torch.where(bad[:, None], 0.0, y2))
