"""Steps over rows of block scores that are longer than the select pass keeps in shared memory, where
the scores behind the buffer decide the result: the blocks there hold a topic of their own, which half of the
heads point at, and values of their own.  Outputs against the fp64 oracle, and the numbers of selected blocks
against its block sets (a block whose score lies within 1e-4 of the threshold may go either way)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import BAND
from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from test_cache8_gpu import close, filled, i32
from test_tree_gpu import path_of

gpu = pytest.mark.gpu
CS, BLK = 0.05, 64


def long_cache(Hq, Hkv, T, d, edge, seed, n=1):
    """q [Hq, n, d] and k, v [1, Hkv, T, d]: blocks from `edge` on have topic 0 and values around 4."""
    g = torch.Generator().manual_seed(seed)
    topics = 2.0 * torch.randn(4, d, generator=g)
    block = torch.randint(1, 4, ((T + BLK - 1) // BLK,), generator=g)
    block[edge:] = 0
    k = topics[block].repeat_interleave(BLK, 0)[:T] + torch.randn(Hkv, T, d, generator=g)
    v = torch.randn(Hkv, T, d, generator=g)
    v[:, edge * BLK:] += 4.0
    q = topics[[h % 2 for h in range(Hq)]].unsqueeze(1) + 0.5 * torch.randn(Hq, n, d, generator=g)
    return q.bfloat16(), k.bfloat16()[None], v.bfloat16()[None], topics, g


def block_sets(q, k, t, Hq):
    """For each head of the row at position t: the blocks that are selected for certain, and those that may be."""
    s = oracle.select_rows(q, k, [(0, h, t) for h in range(Hq)], Hq, BLK, 1.5, CS)
    past = np.arange(s["x"].shape[1])[None] < s["bt"][:, None]
    gap = s["x"] - s["tau"][:, None]
    return past & (gap > BAND), past & (gap > -BAND)


def check_counts(stats, sets, groups):
    """selected_pairs and union_blocks lie between those of the certain and of the possible blocks; rows of
    a group share one list."""
    for i, below in ((0, False), (1, True)):
        pairs = sum(int(s[i].sum()) for s in sets)
        union = sum(int(np.any([sets[r][i] for r in rows], axis=0).sum()) for rows in groups)
        for have, want in ((stats["selected_pairs"], pairs), (stats["union_blocks"], union)):
            assert have <= want if below else have >= want, (stats, pairs, union)


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("Hq,extra", [(8, 0), (5, 40)])
def test_decode_where_the_rest_of_a_row_decides(Hq, extra, q8):
    """8 heads keep 6,656 scores each, 5 heads 10,624 (208 KB a CTA)."""
    d, edge = 64, 208 * 1024 // 4 // Hq // 32 * 32
    T = (edge + 130) * BLK + (0 if q8 else extra)
    L = T - 7
    q, k, v, _, _ = long_cache(Hq, 1, T, d, edge, 301 + Hq)
    v[:, :, (L - 1) // BLK * BLK:] -= 4.0                            # not the own block: it is attended in any case
    q = q[:, 0].contiguous()[None]
    if q8:
        c = filled(1, 1, T, d, k, v)
        k, v = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
        out, ws = da.dash_decode_q8(q.cuda(), *c, i32([L]), coarse_scale=CS)
    else:
        kc = k.cuda()
        out, ws = da.dash_decode(q.cuda(), kc, v.cuda(), da.dash_block_summary(kc), i32([L]), coarse_scale=CS)
    assert da.dash_get_device_status(ws) == 0
    rows = [(0, h, L - 1) for h in range(Hq)]
    ref, _, _ = oracle.forward_rows(q[0], k, v, rows, Hq, BLK, 1.5, CS)
    lost = oracle.fine_rows_given_p(q[0], k, v, rows, Hq, BLK, np.zeros((Hq, T // BLK)), np.ones(Hq))
    assert np.abs(ref - lost)[::2].mean() > 1.0                      # what those heads would give without the rest
    close(out[0].float().cpu(), ref, float(v.float().abs().max()), 1.5, 11 if q8 else 8)
    sure, may = block_sets(q[0], k, L - 1, Hq)
    assert sure[::2, edge:].sum(1).min() > 100 and not may[::2, :edge].any()
    check_counts(da.dash_decode_stats(ws), list(zip(sure, may)), [range(Hq)])


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_trees_where_the_rest_of_a_row_decides(d, q8):
    """A tree step keeps 4,096 scores of a row.  The paths complete one more block, which is selected too."""
    Hq, Hkv, N, edge = 4, 1, 4, 4096
    parent = [-1, 0, 1, 0]
    T, L = (edge + 40) * BLK, (edge + 38) * BLK + 62
    q, k, v, topics, g = long_cache(Hq, Hkv, T, d, edge, 311, n=N)
    kd = (topics[0] + torch.randn(Hkv, N, d, generator=g)).bfloat16()
    vd = torch.randn(Hkv, N, d, generator=g).bfloat16()
    args = (q[None].cuda(), kd[None].cuda(), vd[None].cuda(), i32([parent]))
    if q8:
        c = filled(1, Hkv, T, d, k, v)
        k, v = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
        out, ws = da.dash_decode_tree_q8(*args, *c, i32([L]), coarse_scale=CS)
    else:
        kc = k.cuda()
        out, ws = da.dash_decode_tree(*args, kc, v.cuda(), da.dash_block_summary(kc), i32([L]), coarse_scale=CS)
    assert da.dash_get_device_status(ws) == 0
    sets, full, vmax = [], L // BLK, float(v.float().abs().max())
    for i in range(N):
        p = path_of(parent, i)
        kk, vv = torch.cat((k[:, :, :L], kd[None][:, :, p]), 2).contiguous(), torch.cat((v[:, :, :L], vd[None][:, :, p]), 2).contiguous()
        t = L + len(p) - 1
        rows, qi = [(0, h, t) for h in range(Hq)], q[:, i].contiguous()
        ref, _, _ = oracle.forward_rows(qi, kk, vv, rows, Hq, BLK, 1.5, CS)
        close(out[0, :, i].float().cpu(), ref, vmax, 1.5, 8, f"node {i}")
        nb = kk.shape[2] // BLK
        lost = oracle.fine_rows_given_p(qi, kk, vv, rows, Hq, BLK, np.zeros((Hq, nb)), np.ones(Hq))
        assert np.abs(ref - lost)[::2].mean() > 1.0 or t // BLK == full
        sure, may = block_sets(qi, kk, t, Hq)
        assert sure[::2, edge:].sum(1).min() >= 20 and not may[::2, :edge].any()
        if t // BLK > full:
            assert sure[::2, full].all()                             # the block that the path completes
        wide = np.zeros((2, Hq, full + 1), bool)
        wide[0, :, :sure.shape[1]], wide[1, :, :may.shape[1]] = sure[:, :full + 1], may[:, :full + 1]
        sets += list(zip(wide[0], wide[1]))
    # the open block has an entry of its own in a tile's list
    stats = da.dash_decode_stats(ws)
    pairs = [sum(int(s[i].sum()) for s in sets) for i in (0, 1)]
    union = [int(np.any([s[i][:full] for s in sets], axis=0).sum()) for i in (0, 1)]
    assert pairs[0] <= stats["selected_pairs"] <= pairs[1] and union[0] <= stats["union_blocks"] <= union[1], (stats, pairs, union)
