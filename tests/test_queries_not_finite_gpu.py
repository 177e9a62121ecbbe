"""A query that is no number makes its row NaN and nothing else: the other rows are right, and the device
status of the step stays clean, whatever the bad element meets in the keys."""
import math

import pytest
import torch

import oracle
from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import close, filled, i32
from test_tree_gpu import CS, drafts, expected

gpu = pytest.mark.gpu
BAD = [math.nan, math.inf, -math.inf]


@gpu
@pytest.mark.parametrize("alpha", [1.25, 1.5, 2.0])
@pytest.mark.parametrize("bad", BAD)
def test_decode_q8(bad, alpha):
    """The bad element meets keys of either sign, keys of one sign (infinite scores of that sign), zeros."""
    B, Hq, Hkv, T, d = 3, 6, 2, 320, 64
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=3, seed=231)
    k[1, :, :, 5], k[2, :, :, 5] = k[1, :, :, 5].abs() + 0.5, 0.0
    c = filled(B, Hkv, T, d, k, v)
    kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
    q = q4[:, :, 9].contiguous()
    q[:, [1, 5], 5] = bad
    out, ws = da.dash_decode_q8(q.cuda(), *c, i32([T, 300, 64]), alpha=alpha, coarse_scale=CS)
    assert da.dash_get_device_status(ws) == 0
    out, rest = out.float().cpu(), [0, 2, 3, 4]
    assert bool(out[:, [1, 5]].isnan().all())
    for b, L in enumerate((T, 300, 64)):
        rows = [(0, h, L - 1) for h in range(Hq)]
        ref, _, _ = oracle.forward_rows(torch.nan_to_num(q[b]), kh[b:b + 1], vh[b:b + 1], rows, Hq, 64, alpha, CS)
        close(out[b, rest], ref[rest], float(vh.float().abs().max()), alpha, 11, f"L={L}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", BAD)
def test_trees(bad, q8):
    B, Hq, Hkv, T, d, N = 3, 4, 2, 320, 64, 5
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=3, seed=241)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 242, n_topics=3)
    k[1, :, :, 5], k[2, :, :, 5] = k[1, :, :, 5].abs() + 0.5, 0.0
    kd[1, :, :, 5], kd[2, :, :, 5] = kd[1, :, :, 5].abs() + 0.5, 0.0
    q[:, 1, 2, 5] = bad
    lens, parent = [T, 190, 64], [-1, 0, 1, 2, 0]
    if q8:
        c = filled(B, Hkv, T, d, k, v)
        kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
        out, ws = da.dash_decode_tree_q8(q.cuda(), kd.cuda(), vd.cuda(), i32([parent] * B), *c, i32(lens), coarse_scale=CS)
    else:
        kh, vh = k, v
        out, ws = da.dash_decode_tree(q.cuda(), kd.cuda(), vd.cuda(), i32([parent] * B), k.cuda(), v.cuda(),
                                      da.dash_block_summary(k.cuda()), i32(lens), coarse_scale=CS)
    assert da.dash_get_device_status(ws) == 0
    out = out.float().cpu()
    vmax = float(max(vh.float().abs().max(), vd.float().abs().max()))
    for b, L in enumerate(lens):
        assert bool(out[b, 1, 2].isnan().all())
        ref = expected(torch.nan_to_num(q[b]), kd[b], vd[b], parent, kh[b], vh[b], L, 1.5)
        out[b, 1, 2] = torch.from_numpy(ref[1, 2])
        close(out[b], ref, vmax, 1.5, 8, f"L={L}")
