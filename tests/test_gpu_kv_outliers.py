"""Attention over the 8-bit K/V tile cache with query rows of which a few
channels are far larger than the rest. Both kernels take q as a sum of e4m3
parts of a row that is scaled by its largest value: two parts (more than 16
rows per K/V head) leave out up to 2^-17 of it, four up to 2^-29. The bounds
are those of test_gpu_kv_cache.check_attention, where Q = scale * max |q| *
sum |k| carries that term."""
import pytest
import torch

from tests.test_gpu_kv_cache import bf16, check_attention, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ratio", [8, 11, 14])
@pytest.mark.parametrize("n,heads", [(1, 4), (8, 4), (9, 4), (70, 2), (300, 2)])
@pytest.mark.parametrize("d,tile", [(64, 64), (128, 128)])
def test_channels_far_larger_than_the_others(n, heads, d, tile, ratio):
    """The large channels meet K channels that are zero, so the others decide
    the logits."""
    B, hkv = 2, 2
    c = random_cache(50 + ratio, B, hkv, d, tile, -(-(400 + n) // tile), [400 + n, 150 + n])
    c.len.sub_(n)
    c.next_pos.sub_(n)
    c.k8.view(torch.uint8)[:, :, [3, d - 2]] = 0        # of the tokens that count, and of those behind
    q = bf16(51, B, n, heads, d)
    q[..., [3, d - 2]] *= 2.0 ** ratio
    check_attention(c, q, window=200, sinks=3)
    check_attention(c, q, causal=False, decay=0.0)
