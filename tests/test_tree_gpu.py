"""dash_decode_tree and dash_decode_tree_q8 on the GPU: every node against the fp64 oracle on the
sequence that its path makes (cached tokens, then the path's), and the serving steps together."""
import numpy as np
import pytest
import torch

import oracle
from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import close, filled, i32, junk_cache

gpu = pytest.mark.gpu
CS = 0.05


def path_of(parent, i):
    p = [i]
    while parent[p[0]] >= 0:
        p.insert(0, parent[p[0]])
    return p


def random_tree(N, seed, width=3):
    g = np.random.RandomState(seed)
    return [int(max(-1, i - 1 - g.randint(0, width))) if i else -1 for i in range(N)]


def expected(q, kd, vd, parent, k, v, L, alpha, nodes=None):
    """fp64 rows of one sequence: q [Hq, N, d], drafts [Hkv, N, d], cache [Hkv, T, d]."""
    Hq, N, d = q.shape
    ref = np.zeros((Hq, N, d))
    for i in range(N if nodes is None else nodes):
        p = path_of(parent, i)
        ks, vs = torch.cat((k[:, :L], kd[:, p]), 1)[None], torch.cat((v[:, :L], vd[:, p]), 1)[None]
        t = L + len(p) - 1
        out, _, _ = oracle.forward_rows(q[:, i].contiguous(), ks.contiguous(), vs.contiguous(), [(0, h, t) for h in range(Hq)], Hq, 64, alpha, CS)
        ref[:, i] = out
    return ref


def drafts(B, Hq, Hkv, N, d, seed, n_topics=4):
    _, (q, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=N, d=d, n_topics=n_topics, seed=seed)
    return q, k, v


def run(q8, q, kd, vd, parent, k, v, lens, alpha, n_nodes=None, out=None, junk=True):
    """The call on the GPU; returns its output and the cache values that it used."""
    B, Hkv, T, d = k.shape
    if q8:
        c = junk_cache(B, Hkv, T, d)
        da.dash_cache_append(k.cuda(), v.cuda(), i32([0] * B), *c[:4], ksum=c[4], n=T, n_new=i32([max(0, min(T, x)) for x in lens]))
        kh, vh = da.dash_cache_read(*c[:4], T, kv_len=i32([max(0, min(T, x)) for x in lens]))
        got, ws = da.dash_decode_tree_q8(q.cuda(), kd.cuda(), vd.cuda(), i32(parent), *c[:4], c[4], i32(lens), alpha=alpha,
                                         coarse_scale=CS, n_nodes=n_nodes, out=out)
        kh, vh = kh.cpu(), vh.cpu()
    else:
        kh, vh = k, v
        kc, vc = k.cuda(), v.cuda()
        ksum = da.dash_block_summary(kc)
        if junk:                                                     # rows behind a sequence are not used
            for b, L in enumerate(lens):
                kc[b, :, max(0, L):] = float("nan")
                vc[b, :, max(0, L):] = float("inf")
        got, ws = da.dash_decode_tree(q.cuda(), kd.cuda(), vd.cuda(), i32(parent), kc, vc, ksum, i32(lens), alpha=alpha,
                                      coarse_scale=CS, n_nodes=n_nodes, out=out)
    assert da.dash_get_device_status(ws) == 0
    return got, kh, vh


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,N,alpha", [(1, 1, 64, 1, 1.5), (4, 2, 128, 5, 1.5), (8, 1, 64, 17, 2.0), (6, 2, 128, 33, 1.25),
                                              (16, 1, 64, 9, 1.5), (3, 1, 128, 64, 1.5), (32, 1, 64, 6, 3.0)])
def test_tree_against_oracle(Hq, Hkv, d, N, alpha, q8):
    lens = [0, 1, 63, 64, 300, 384]
    B, T = len(lens), 384
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=4, seed=41 + N)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 43 + N)
    parent = [random_tree(N, 7 * b + N) for b in range(B)]
    got, kh, vh = run(q8, q, kd, vd, parent, k, v, lens, alpha)
    vmax = float(max(vh.float().abs().max(), vd.float().abs().max()))
    for b in range(B):
        ref = expected(q[b], kd[b], vd[b], parent[b], kh[b], vh[b], lens[b], alpha)
        close(got[b].float().cpu(), ref, vmax, alpha, 8, f"L={lens[b]}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_long_path_over_the_end_of_a_block(q8):
    """A chain of 64: for each start in the open block some nodes complete it; a star never does."""
    lens = [1, 32, 63, 127, 200, 256]
    B, Hq, Hkv, T, d, N = len(lens), 4, 2, 256, 64, 64
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=3, seed=51)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 52, n_topics=3)
    for parent in ([list(range(-1, N - 1))] * B, [[-1] * N] * B, [[-1] + [max(0, (i - 1) // 2) for i in range(1, N)]] * B):
        got, kh, vh = run(q8, q, kd, vd, parent, k, v, lens, 1.5)
        vmax = float(max(vh.float().abs().max(), vd.float().abs().max()))
        for b in range(B):
            ref = expected(q[b], kd[b], vd[b], parent[b], kh[b], vh[b], lens[b], 1.5)
            close(got[b].float().cpu(), ref, vmax, 1.5, 8, f"L={lens[b]}")


@gpu
def test_bf16_cache_of_any_length():
    """Tmax that ends inside a block, and caches shorter than a block."""
    for T, lens in ((40, [40, 7]), (100, [100, 64]), (321, [321, 320])):
        B, Hq, Hkv, d, N = 2, 4, 1, 128, 12
        _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=3, seed=61)
        q, kd, vd = drafts(B, Hq, Hkv, N, d, 62, n_topics=3)
        parent = [random_tree(N, b) for b in range(B)]
        got, kh, vh = run(False, q, kd, vd, parent, k, v, lens, 1.5)
        for b in range(B):
            ref = expected(q[b], kd[b], vd[b], parent[b], kh[b], vh[b], lens[b], 1.5)
            close(got[b].float().cpu(), ref, float(v.float().abs().max()), 1.5, 8, f"T={T} L={lens[b]}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_padded_nodes_bad_parents_and_bad_lengths(q8):
    B, Hq, Hkv, T, d, N = 6, 4, 2, 128, 64, 8
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=71)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 72, n_topics=2)
    parent = [random_tree(N, b) for b in range(B)]
    parent[1] = [-1, 0, 5, 2, 1, -2, 5, 4]                           # 2 and 5 invalid; 3 and 6 descend from them
    parent[2] = [-1, 0, 1] + [99] * 5                                # padded with anything
    lens = [100, 100, 70, -1, 129, 64]
    n_nodes = [8, 8, 3, 8, 8, 0]
    kd[2, :, 3:] = float("nan")                                      # rows of nodes that are not there
    vd[2, :, 3:] = float("inf")
    mark = torch.full((B, Hq, N, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got, kh, vh = run(q8, q, kd, vd, parent, k, v, lens, 1.5, n_nodes=i32(n_nodes), out=mark)
    got = got.float().cpu()
    assert bool((got[3] == 0).all()) and bool((got[4] == 0).all())   # lengths outside [0, Tmax]
    assert bool((got[5] == 3).all()) and bool((got[2][:, 3:] == 3).all())
    assert bool((got[1][:, [2, 3, 5, 6]] == 0).all())
    vmax = float(vh.float().abs().max()) + 4.0
    for b, live in ((0, range(8)), (1, [0, 1, 4, 7]), (2, [0, 1, 2])):
        pa = [p if i in live else -1 for i, p in enumerate(parent[b])]
        ref = expected(q[b], torch.nan_to_num(kd[b]), torch.nan_to_num(vd[b]), pa, kh[b], vh[b], lens[b], 1.5)
        close(got[b][:, list(live)], ref[:, list(live)], vmax, 1.5, 8, f"sequence {b}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_many_rows_and_long_lists(q8):
    """More rows than a tile, and lists split over CTAs: sampled nodes against the oracle."""
    B, Hq, Hkv, T, d, N = 2, 16, 2, 8192, 128, 40
    lens = [8192, 5003]
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=8, seed=81)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 82, n_topics=8)
    parent = [random_tree(N, 3), list(range(-1, N - 1))]
    got, kh, vh = run(q8, q, kd, vd, parent, k, v, lens, 1.5)
    vmax = float(vh.float().abs().max())
    for b in range(B):
        for i in (0, 1, 20, N - 1):
            p = path_of(parent[b], i)
            ks, vs = torch.cat((kh[b, :, :lens[b]], kd[b][:, p]), 1)[None], torch.cat((vh[b, :, :lens[b]], vd[b][:, p]), 1)[None]
            t = lens[b] + len(p) - 1
            ref, _, _ = oracle.forward_rows(q[b, :, i].contiguous(), ks.contiguous(), vs.contiguous(), [(0, h, t) for h in range(Hq)], Hq, 64, 1.5, CS)
            close(got[b, :, i].float().cpu(), ref, vmax, 1.5, 8, f"sequence {b} node {i}")


@gpu
def test_serving_steps_together():
    """Prompt appended, a drafted tree attended, its accepted path appended by index, the next token's
    step: each against the oracle on what the cache holds; on a stream of its own, then from a graph."""
    B, Hq, Hkv, d, N, T = 2, 8, 2, 128, 6, 256
    _, (qs, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=130, d=d, n_topics=3, seed=91)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 92, n_topics=3)
    lens = [126, 61]
    parent = [[-1, 0, 1, 1, 3, 4], [-1, 0, 0, 2, 3, 3]]
    src, n_new = i32([[0, 1, 3, 4], [0, 2, 3, 0]]), i32([4, 3])
    q1 = qs[:, :, 7].contiguous()
    kq, vq, qg, kdg, vdg, q1g = k.cuda(), v.cuda(), q.cuda(), kd.cuda(), vd.cuda(), q1.cuda()
    cache = junk_cache(B, Hkv, T, d)
    par, start, zero = i32(parent), i32(lens), i32([0, 0])
    out_t, out_1 = torch.empty_like(qg), torch.empty_like(q1g)
    ws_t = da.alloc_workspace(da.decode_tree_workspace_size(B, Hq, Hkv, N, T, d))
    ws_1 = da.alloc_workspace(da.decode_q8_workspace_size(B, Hq, Hkv, T, d))
    after = start + n_new

    def step():
        da.dash_cache_append(kq, vq, zero, *cache[:4], ksum=cache[4], n_new=start, n=130)
        da.dash_decode_tree_q8(qg, kdg, vdg, par, *cache[:4], cache[4], start, out=out_t, coarse_scale=CS, workspace=ws_t)
        da.dash_cache_append(kdg, vdg, start, *cache[:4], ksum=cache[4], src=src, n_new=n_new)
        da.dash_decode_q8(q1g, *cache, after, out=out_1, coarse_scale=CS, workspace=ws_1)

    def check():
        kh, vh = (x.cpu() for x in da.dash_cache_read(*cache[:4], T, kv_len=after))
        vmax = float(max(vh.float().abs().max(), vd.float().abs().max()))
        for b in range(B):
            ref = expected(q[b], kd[b], vd[b], parent[b], kh[b], vh[b], lens[b], 1.5)
            close(out_t[b].float().cpu(), ref, vmax, 1.5, 8, f"tree {b}")
        rws = [(b, h, int(after[b]) - 1) for b in range(B) for h in range(Hq)]
        ref, _, _ = oracle.forward_rows(q1.reshape(-1, d), kh, vh, rws, Hq, 64, 1.5, CS)
        close(out_1.float().cpu().reshape(-1, d), ref, vmax, 1.5, 11, "step")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check()
    first = [out_t.clone(), out_1.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        for t in (out_t, out_1):
            t.fill_(9.0)
        for t in cache[:4]:
            t.view(torch.uint8).fill_(0x7f)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_t, first[0]) and torch.equal(out_1, first[1])
    del g
    check()


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_more_tiles_than_a_merge_adds_up(q8):
    """From 1024 lists on, the merge looks its pieces up in what the attention left."""
    B, Hq, Hkv, T, d, N = 520, 4, 2, 128, 64, 3
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=101)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 102, n_topics=2)
    parent = [[-1, 0, 0] if b % 2 else [-1, 0, 1] for b in range(B)]
    lens = [(37 * b) % 129 for b in range(B)]
    got, kh, vh = run(q8, q, kd, vd, parent, k, v, lens, 1.5, junk=False)
    got = got.float().cpu()
    for b in [0, 1, 2, 7, 100, 255, 256, 511, 512, 518, 519] + [b for b in range(B) if lens[b] in (0, 63, 64, 128)][:8]:
        ref = expected(q[b], kd[b], vd[b], parent[b], kh[b], vh[b], lens[b], 1.5)
        close(got[b], ref, float(max(v[b].float().abs().max(), vd[b].float().abs().max())) * 1.1, 1.5, 8, f"sequence {b}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_rows_longer_than_the_shared_buffer(q8):
    """More blocks than a warp keeps in shared memory (4096), where the paths complete one more."""
    B, Hq, Hkv, T, d, N = 1, 2, 1, 262144 + 640, 64, 3
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=8, seed=111)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 112, n_topics=8)
    for L in (T - 1, 262144 + 63):
        got, kh, vh = run(q8, q, kd, vd, [[-1, 0, 1]], k, v, [L], 1.5, junk=False)
        ref = expected(q[0], kd[0], vd[0], [-1, 0, 1], kh[0], vh[0], L, 1.5)
        close(got[0].float().cpu(), ref, float(v.float().abs().max()) * 1.1, 1.5, 8, f"L={L}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_key_that_is_no_number_stays_on_its_paths(q8, bad):
    """Node 5's key is no number: nodes that do not descend from it are right, in the open block (L = 10)
    and where paths complete it (L = 61), whose summaries must not take it up either."""
    B, Hq, Hkv, T, d, N = 2, 4, 2, 128, 64, 12
    lens = [10, 61]
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=121)
    q, kd, vd = drafts(B, Hq, Hkv, N, d, 122, n_topics=2)
    parent = [-1, 0, 1, 2, 3, 1, 5, 4, 7, 6, 8, 10]
    others = [0, 1, 2, 3, 4, 7, 8, 10, 11]
    kd[:, :, 5, 3] = bad
    got, kh, vh = run(q8, q, kd, vd, [parent] * B, k, v, lens, 1.5)
    clean = torch.where(torch.isfinite(kd), kd, torch.zeros_like(kd))
    for b in range(B):
        ref = expected(q[b], clean[b], vd[b], parent, kh[b], vh[b], lens[b], 1.5)
        vmax = float(max(v[b].float().abs().max(), vd[b].float().abs().max())) * 1.1
        close(got[b].float().cpu()[:, others], ref[:, others], vmax, 1.5, 8, f"L={lens[b]}")


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_two_trees_at_once_from_graphs_with_any_workspace(q8):
    """Two captured steps replayed on two streams, with workspaces of their own that held anything, give
    what each gives alone, bit for bit; rows of another sequence's values that are NaN reach no one else."""
    Hq, Hkv, d = 8, 2, 128
    sides = []
    for T, N, seed in ((4096, 16, 131), (2048, 40, 132)):
        _, (_, k, v) = inputs.make("16k", B=2, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=4, seed=seed)
        q, kd, vd = (x.cuda() for x in drafts(2, Hq, Hkv, N, d, seed + 5))
        par, lens = i32([random_tree(N, seed), list(range(-1, N - 1))]), i32([T, T - 70])
        v[1, 0, 3] = float("nan")
        if q8:
            c = filled(2, Hkv, T, d, k, v)
            args = (q, kd, vd, par, *c[:4], c[4], lens)
            fn = da.dash_decode_tree_q8
        else:
            kc = k.cuda()
            args = (q, kd, vd, par, kc, v.cuda(), da.dash_block_summary(kc), lens)
            fn = da.dash_decode_tree
        alone, ws = fn(*args, coarse_scale=CS)
        assert bool(torch.isfinite(alone[0]).all())
        ws, out = torch.full_like(ws, 255), torch.empty_like(alone)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fn(*args, coarse_scale=CS, workspace=ws, out=out)
        sides.append((graph, torch.cuda.Stream(), out, alone, args, ws))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, stream, out, *_ in sides:
            with torch.cuda.stream(stream):
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, _, out, alone, *_ in sides:
            assert torch.equal(out.view(torch.int16), alone.view(torch.int16))


@gpu
def test_refusals_with_gpu_tensors_and_a_stream_argument():
    B, Hq, Hkv, T, d, N = 2, 4, 2, 128, 64, 4
    _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=141)
    q, kd, vd = (x.cuda() for x in drafts(B, Hq, Hkv, N, d, 142, n_topics=2))
    c, par, lens = filled(B, Hkv, T, d, k, v), i32([[-1, 0, 1, 0]] * B), i32([100, 64])
    call = lambda *a, **kw: da.dash_decode_tree_q8(*a, coarse_scale=CS, **kw)  # noqa: E731
    good = [q, kd, vd, par, *c, lens]
    want, ws = call(*good)
    for i, bad in ((0, q.transpose(1, 2)), (0, q.float()), (1, kd[:, :1]), (3, par.long()), (4, c[0].view(torch.uint8)),
                   (6, c[2][:, :, :64]), (8, c[4].half()), (9, lens.cpu()), (9, lens[:1])):
        with pytest.raises(ValueError):
            call(*good[:i], bad, *good[i + 1:])
    with pytest.raises(ValueError):
        call(*good, out=torch.empty_like(q).transpose(0, 1).contiguous())
    with pytest.raises(ValueError):
        call(*good, workspace=ws.cpu())
    for small in (ws[:-256], ws[16:]):                               # too small, not aligned
        with pytest.raises(da.DashError):
            call(*good, workspace=small)
    with pytest.raises(da.DashError):
        da.dash_decode_tree_q8(*good, alpha=1.0)
    side, out = torch.cuda.Stream(), torch.full_like(want, 9.0)
    side.wait_stream(torch.cuda.current_stream())
    call(*good, out=out, workspace=ws, stream=side)
    k1, _ = da.dash_cache_read(*c[:4], T, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(k1, da.dash_cache_read(*c[:4], T)[0])
