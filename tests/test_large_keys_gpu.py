"""Keys near the largest number that the 8-bit cache holds: the summaries of blocks, and of blocks that a
drafted path completes, are their means, which are numbers although the keys' sum is not one in fp32."""
import pytest
import torch

import oracle
from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import close, filled, i32, junk_cache
from test_tree_gpu import drafts, expected, run

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


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("where", ["cache", "draft", "both"])
def test_paths_that_complete_a_block_of_large_keys(q8, where):
    """The open block's keys hold bf16's largest numbers in a dim that no query has: scores and outputs are
    those of the other dims."""
    B, Hq, Hkv, T, d, N, dim = 1, 4, 2, 192, 64, 8, 11
    L, parent = 128 + 59, [-1, 0, 1, 2, 3, 4, 5, 5]
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=91)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 92, n_topics=2)
    q[..., dim] = 0.0
    if where != "draft":
        k[:, :, 128:140, dim] = 240.0 * 2.0 ** 120
    if where != "cache":
        kd[:, :, 1:4, dim] = 240.0 * 2.0 ** 120
    got, kh, vh = run(q8, q, kd, vd, [parent], k, v, [L], 1.5, junk=False)
    ref = expected(q[0], kd[0], vd[0], parent, kh[0], vh[0], L, 1.5)
    close(got[0].float().cpu(), ref, float(max(vh.float().abs().max(), vd.float().abs().max())), 1.5, 8, where)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_decode_q8_large_keys_beside_large_queries(d):
    """Keys of 2^110 in a dim that the query lacks, queries of 2^40 in one that the keys lack: every logit is
    zero, though the key's and the query's scales multiply to no finite number."""
    B, Hq, Hkv, T = 1, 4, 2, 192
    g = torch.Generator().manual_seed(29)
    k, v = torch.randn(B, Hkv, T, d, generator=g), torch.randn(B, Hkv, T, d, generator=g)
    q = torch.zeros(B, Hq, d)
    k[..., 7], q[..., 7] = 0.0, 2.0 ** 40
    for t in (5, 70, 150):
        k[:, :, t, 3] = 2.0 ** 110
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    c = filled(B, Hkv, T, d, k, v)
    kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
    out, ws = da.dash_decode_q8(q.cuda(), *c, i32([T]), coarse_scale=0.05)
    assert da.dash_get_device_status(ws) == 0
    ref, _, _ = oracle.forward_rows(q[0], kh, vh, [(0, h, T - 1) for h in range(Hq)], Hq, 64, 1.5, 0.05)
    close(out[0].float().cpu(), ref, float(vh.float().abs().max()), 1.5, 11)
