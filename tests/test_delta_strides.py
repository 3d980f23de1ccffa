"""How the gated delta rule's binding takes q, k and v: tokens one stride apart,
which the library must never see shorter than a token's heads (0 would mean
dense to it). On the CPU."""
import pytest
import torch

from self_referential_memory_amd import srnl


@pytest.mark.parametrize("src,shape", [
    # one token for all: over items and tokens, over the tokens of one item, over items
    ((1, 1, 2, 16), (3, 5, 2, 16)), ((1, 1, 2, 16), (1, 5, 2, 16)), ((1, 1, 2, 16), (3, 1, 2, 16)),
    # one item for all, one token an item, one head for all
    ((1, 5, 2, 16), (3, 5, 2, 16)), ((3, 1, 2, 16), (3, 5, 2, 16)), ((3, 5, 1, 16), (3, 5, 2, 16))])
def test_broadcast_views_are_refused(src, shape):
    with pytest.raises(ValueError, match="q must be contiguous"):
        srnl._token_stride(torch.zeros(src).expand(shape), "q")


@pytest.mark.parametrize("step", [8, 24, 31])
@pytest.mark.parametrize("B,T", [(1, 5), (3, 1), (3, 5)])
def test_overlapping_tokens_are_refused(B, T, step):
    t = torch.zeros(B * T * step + 32).as_strided((B, T, 2, 16), (T * step, step, 16, 1))
    with pytest.raises(ValueError, match="k must be contiguous"):
        srnl._token_stride(t, "k")


@pytest.mark.parametrize("B,T", [(1, 5), (3, 1), (3, 5), (1, 1)])
def test_slices_and_dense_tensors_are_taken(B, T):
    assert srnl._token_stride(torch.zeros(B, T, 2, 16), "v") == 0
    p = torch.zeros(B, T, 40)[..., 8:].unflatten(2, (2, 16))
    assert srnl._token_stride(p, "v") == (0 if B * T == 1 else 40)
    dense = torch.zeros(B * T * 32).as_strided((B, T, 2, 16), (T * 32, 32, 16, 1))
    assert srnl._token_stride(dense, "v") == 0


def test_one_head_of_a_wider_row_is_taken():
    """A single head's stride to the next one says nothing."""
    p = torch.zeros(3, 5, 1, 40)
    assert srnl._token_stride(p[..., 8:24], "q") == 40
    assert srnl._token_stride(p[:, :1].contiguous()[..., 8:24], "q") == 40
    assert srnl._token_stride(torch.zeros(3, 5, 4, 16)[:, :, 1:2], "q") == 64
    with pytest.raises(ValueError, match="q must be contiguous"):
        srnl._token_stride(torch.zeros(3, 5, 2, 40)[..., 8:24], "q")
