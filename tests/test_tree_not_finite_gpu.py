"""dash_decode_tree and dash_decode_tree_q8: a key that is no number makes every row that attends it NaN,
also where it is the only key that the row attends in a 64-key entry."""
import math

import pytest
import torch

from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import close, filled, i32
from test_tree_gpu import CS, drafts, expected, path_of

gpu = pytest.mark.gpu


def step(q8, q, kd, vd, parent, k, v, lens, ksum=None):
    """The call on [B, Hkv, T, d] caches; returns its output, and the cache values that it used."""
    B, Hkv, T, d = k.shape
    if q8:
        c = filled(B, Hkv, T, d, k, v)
        kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
        if ksum is not None:
            c[4].copy_(ksum)
        out, ws = da.dash_decode_tree_q8(q.cuda(), kd.cuda(), vd.cuda(), i32(parent), *c, i32(lens), coarse_scale=CS)
    else:
        kh, vh = k, v
        ks = da.dash_block_summary(k.cuda()) if ksum is None else ksum.cuda()
        out, ws = da.dash_decode_tree(q.cuda(), kd.cuda(), vd.cuda(), i32(parent), k.cuda(), v.cuda(), ks, i32(lens), coarse_scale=CS)
    assert da.dash_get_device_status(ws) == 0
    return out.float().cpu(), kh, vh


def rows(B, Hq, Hkv, T, d, N, seed):
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=seed)
    return (k, v, *drafts(B, Hq, Hkv, N, d, seed + 1, n_topics=2))


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [0, 2, 5])
def test_a_drafted_key_that_is_nan_reaches_its_node_and_its_descendants(q8, d, bad):
    """Node 0 and node 5 are roots: their own key is all that they attend of the draft."""
    lens = [0, 1, 40, 61, 64, 192]
    B, Hq, Hkv, T, N = len(lens), 4, 2, 192, 8
    parent = [-1, 0, 1, 2, 0, -1, 5, 6]
    k, v, q, kd, vd = rows(B, Hq, Hkv, T, d, N, 201)
    kd[:, :, bad, 7] = math.nan
    out, kh, vh = step(q8, q, kd, vd, [parent] * B, k, v, lens)
    hit = [i for i in range(N) if bad in path_of(parent, i)]
    rest = [i for i in range(N) if i not in hit]
    clean = torch.nan_to_num(kd)
    vmax = float(max(vh.float().abs().max(), vd.float().abs().max()))
    for b, L in enumerate(lens):
        assert bool(out[b][:, hit].isnan().all()), f"L={L}"
        ref = expected(q[b], clean[b], vd[b], parent, kh[b], vh[b], L, 1.5)
        close(out[b][:, rest], ref[:, rest], vmax, 1.5, 8, f"L={L}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_an_open_block_whose_keys_are_nan_reaches_every_row(q8):
    """One cached token in the open block, and three; a tree of one node, and of four."""
    for N, parent in ((1, [-1]), (4, [-1, 0, -1, 2])):
        B, Hq, Hkv, T, d = 2, 4, 2, 192, 64
        k, v, q, kd, vd = rows(B, Hq, Hkv, T, d, N, 211)
        ksum = da.dash_block_summary(k.cuda())
        lens = [65, 131]
        k[0, 0, 64], k[1, 0, 128:131] = math.nan, math.nan
        out, kh, vh = step(q8, q, kd, vd, [parent] * B, k, v, lens, ksum)
        G = Hq // Hkv
        assert bool(out[:, :G].isnan().all())
        kz, vmax = torch.nan_to_num(kh), float(max(torch.nan_to_num(vh).float().abs().max(), vd.float().abs().max()))
        for b in range(B):
            ref = expected(q[b], kd[b], vd[b], parent, kz[b], vh[b], lens[b], 1.5)
            close(out[b, G:], ref[G:], vmax, 1.5, 8, f"N={N}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T,L", [(256, 200), (8192, 8192 - 8)])
def test_a_past_block_whose_keys_are_all_nan_reaches_the_rows_that_select_it(q8, T, L):
    """Heads 0 and 1 point at blocks 0 and 1; block 0's keys become NaN, its summary stays.  The longer
    cache's lists are split over CTAs."""
    B, Hq, Hkv, d, N = 1, 2, 1, 64, 2
    g = torch.Generator().manual_seed(7)
    k, v = torch.zeros(B, Hkv, T, d), torch.randn(B, Hkv, T, d, generator=g).bfloat16()
    q = torch.zeros(B, Hq, N, d)
    for j in range(2):
        k[:, :, 64 * j:64 * j + 64, j] = 4.0
        q[:, j, :, j] = 400.0
    kd, vd = torch.zeros(B, Hkv, N, d).bfloat16(), torch.randn(B, Hkv, N, d, generator=g).bfloat16()
    k = k.bfloat16()
    ksum = da.dash_block_summary(k.cuda())
    for part in (slice(0, 64), slice(3, 4)):                         # all keys, and one beside 63 numbers
        k2 = k.clone()
        k2[:, :, part] = math.nan
        out, _, vh = step(q8, q.bfloat16(), kd, vd, [[-1, -1]], k2, v, [L], ksum)
        assert bool(out[:, 0].isnan().all())
        vmax = float(max(vh.float().abs().max(), vd.float().abs().max()))
        ref = expected(q.bfloat16()[0], kd[0], vd[0], [-1, -1], k[0], vh[0], L, 1.5)
        close(out[0, 1], ref[1], vmax, 1.5, 8)
