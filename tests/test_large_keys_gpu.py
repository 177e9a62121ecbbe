"""Keys near the largest number that the 8-bit cache holds: the summaries are their means, which are numbers
although the keys' sum is not one in fp32."""
import pytest
import torch

from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from test_cache8_gpu import i32, junk_cache

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first", [0, 40])
def test_summaries_of_keys_whose_sum_is_no_number(d, first):
    """Blocks with 2, 33 and 64 large keys of one sign, written at once or as the second part of a block."""
    B, Hkv, T = 1, 2, 192
    g = torch.Generator().manual_seed(17)
    k = torch.randn(B, Hkv, T, d, generator=g)
    top = 240.0 * 2.0 ** 120
    for j, n in enumerate((2, 33, 64)):
        k[:, 0, 64 * j:64 * j + n, 3] = top
        k[:, 1, 64 * j:64 * j + n, 5] = -top * 0.75
    k, v = k.bfloat16().cuda(), torch.zeros(B, Hkv, T, d).bfloat16().cuda()
    c = junk_cache(B, Hkv, T, d)
    if first:
        da.dash_cache_append(k[:, :, :first].contiguous(), v[:, :, :first].contiguous(), i32([0]), *c[:4], ksum=c[4])
    da.dash_cache_append(k[:, :, first:].contiguous(), v[:, :, first:].contiguous(), i32([first]), *c[:4], ksum=c[4])
    held, _ = da.dash_cache_read(*c[:4], T)
    blk = held.double().cpu().view(B, Hkv, 3, 64, d)
    want = blk.mean(3)
    got = c[4].double().cpu()
    assert bool(torch.isfinite(got).all())
    # 64 fp32 additions: off by at most 64 2^-24 of the sum of magnitudes, each a 64th
    assert bool(((got - want).abs() <= 2.0 ** -18 * blk.abs().mean(3)).all())


@gpu
@pytest.mark.parametrize("p", [0, -60, -100, -126])
def test_summaries_of_small_keys(p):
    """Keys down to the least held numbers: a mean's rounding stays that of 64 fp32 additions."""
    B, Hkv, T, d = 1, 1, 64, 64
    g = torch.Generator().manual_seed(19)
    k = (torch.randn(B, Hkv, T, d, generator=g) * torch.exp2(-8 * torch.rand(B, Hkv, T, 1, generator=g))).double()
    k = (k * 2.0 ** p).bfloat16().cuda()
    c = junk_cache(B, Hkv, T, d)
    da.dash_cache_append(k, k, i32([0]), *c[:4], ksum=c[4])
    held = da.dash_cache_read(*c[:4], T)[0].double().cpu()
    # half the least subnormal fp32 where a mean is that small
    tol = 2.0 ** -18 * held.abs().mean(2) + 2.0 ** -150
    assert bool(((c[4][:, :, 0].double().cpu() - held.mean(2)).abs() <= tol).all())
