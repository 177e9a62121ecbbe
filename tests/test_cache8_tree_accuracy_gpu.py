"""The 8-bit step and the tree steps by the specification's tolerances (max-abs 2e-2 and mean-abs 2e-3 against the
fp64 oracle), and by what they select: the counts of scored and selected pairs and of listed blocks against the
oracle's block sets, where a block within 1e-4 of the threshold, and a score's own rounding, may go either way."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import BAND, compare_out, score_allowance
from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import filled, i32
from test_tree_gpu import drafts, path_of, random_tree

gpu = pytest.mark.gpu
BLK, CS = 64, 0.05


def row_sets(q, k, t, Hq, alpha, nb):
    """(certain, possible) blocks [Hq, nb] of every head of the row at position t of one sequence."""
    rows = [(0, h, t) for h in range(Hq)]
    s = oracle.select_rows(q, k, rows, Hq, BLK, alpha, CS)
    band = BAND + score_allowance(q, k, rows, Hq, alpha, CS)[:, None]
    past = np.arange(s["x"].shape[1])[None] < s["bt"][:, None]
    gap = s["x"] - s["tau"][:, None]
    out = np.zeros((2, Hq, nb), bool)
    out[0, :, :past.shape[1]], out[1, :, :past.shape[1]] = past & (gap > band), past & (gap > -band)
    return out, int(s["bt"].sum())


def between(stats, scored, pairs, union):
    assert stats["scored_pairs"] == scored
    assert pairs[0] <= stats["selected_pairs"] <= pairs[1], (stats, pairs)
    assert union[0] <= stats["union_blocks"] <= union[1], (stats, union)


@gpu
@pytest.mark.parametrize("Hq,Hkv,d,alpha", [(16, 2, 128, 1.5), (16, 2, 128, 1.25), (8, 4, 64, 2.0), (24, 2, 128, 1.5), (11, 1, 64, 1.5)])
def test_decode_q8(Hq, Hkv, d, alpha):
    B, T = 3, 4096
    lens = [4096, 2500, 65]
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=16, seed=401 + Hq)
    c = filled(B, Hkv, T, d, k, v)
    kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
    q = q4[:, :, 33].contiguous()
    out, ws = da.dash_decode_q8(q.cuda(), *c, i32(lens), alpha=alpha, coarse_scale=CS)
    assert da.dash_get_device_status(ws) == 0
    G = Hq // Hkv
    part = G // next(s for s in range(1, G + 1) if G % s == 0 and G // s <= 8)     # heads that share a list
    scored, pairs, union = 0, [0, 0], [0, 0]
    for b, L in enumerate(lens):
        rows = [(0, h, L - 1) for h in range(Hq)]
        ref, _, _ = oracle.forward_rows(q[b], kh[b:b + 1], vh[b:b + 1], rows, Hq, BLK, alpha, CS)
        compare_out(out[b].float().cpu(), ref, f"L={L}")
        sets, n = row_sets(q[b], kh[b:b + 1], L - 1, Hq, alpha, T // BLK)
        scored += n
        for i in (0, 1):
            pairs[i] += int(sets[i].sum())
            union[i] += sum(int(sets[i][h:h + part].any(0).sum()) for h in range(0, Hq, part))
    between(da.dash_decode_stats(ws), scored, pairs, union)


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,N,alpha", [(16, 2, 128, 16, 1.5), (8, 2, 128, 5, 1.25), (8, 4, 64, 40, 2.0), (11, 1, 64, 13, 1.5)])
def test_trees(Hq, Hkv, d, N, alpha, q8):
    B, T = 3, 2048
    lens = [2048, 1500 // BLK * BLK + 61, 20]
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=16, seed=421 + N)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 422 + N, n_topics=16)
    parent = [random_tree(N, 5 * b + 1) for b in range(B)]
    args = (q.cuda(), kd.cuda(), vd.cuda(), i32(parent))
    if q8:
        c = filled(B, Hkv, T, d, k, v)
        kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
        out, ws = da.dash_decode_tree_q8(*args, *c, i32(lens), alpha=alpha, coarse_scale=CS)
    else:
        kh, vh = k, v
        out, ws = da.dash_decode_tree(*args, k.cuda(), v.cuda(), da.dash_block_summary(k.cuda()), i32(lens), alpha=alpha, coarse_scale=CS)
    assert da.dash_get_device_status(ws) == 0
    G, scored, pairs, union = Hq // Hkv, 0, [0, 0], [0, 0]
    for b, L in enumerate(lens):
        full, nb = L // BLK, T // BLK + 1
        sets = np.zeros((2, Hq, N, nb), bool)
        ref = np.zeros((Hq, N, d))
        for i in range(N):
            p = path_of(parent[b], i)
            kk, vv = (torch.cat((a[b, :, :L], x[b][:, p]), 1)[None].contiguous() for a, x in ((kh, kd), (vh, vd)))
            t, qi = L + len(p) - 1, q[b, :, i].contiguous()
            ref[:, i], _, _ = oracle.forward_rows(qi, kk, vv, [(0, h, t) for h in range(Hq)], Hq, BLK, alpha, CS)
            sets[:, :, i], n = row_sets(qi, kk, t, Hq, alpha, nb)
            scored += n
        compare_out(out[b].float().cpu(), ref, f"L={L}")
        for i in (0, 1):
            pairs[i] += int(sets[i].sum())
            # tiles of 128 rows (head, node) of a KV head; the open block has an entry of its own
            rows = sets[i][:, :, :full].reshape(Hkv, G * N, full)
            union[i] += sum(int(rows[g, r:r + 128].any(0).sum()) for g in range(Hkv) for r in range(0, G * N, 128))
    between(da.dash_decode_stats(ws), scored, pairs, union)
