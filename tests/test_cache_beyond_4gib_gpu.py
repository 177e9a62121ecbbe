"""Caches whose bytes pass 32-bit offsets: the last KV head, whose rows lie behind 2^32 bytes, gives what it gives in
a cache of its own.  (All other heads' rows are zeros, so an offset that wrapped would find zeros or another head.)"""
import pytest
import torch

from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from test_cache8_gpu import i32, same_bits, weight_error

gpu = pytest.mark.gpu
T, D, H = 1 << 20, 128, 36
CS = 0.05


def near(a, b, vmax, w_bits):
    """Both are off by at most half a bf16 step and twice their weights' error (test_cache8_gpu.close)."""
    a, b = a.double(), b.double()
    tol = 2.0 ** -8 * (a.abs() + b.abs()) + 4 * weight_error(1.5, w_bits) * vmax
    assert bool(((a - b).abs() <= tol).all())
    assert float(b.mean()) > 1.0                                     # far from what zeros would give


def rows(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(1, 1, n, D, device="cuda", generator=g)
    k += 2.0 * torch.randn(8, D, device="cuda", generator=g)[torch.randint(0, 8, ((n + 63) // 64,), device="cuda", generator=g)].repeat_interleave(64, 0)[:n]
    return k.bfloat16(), (torch.randn(1, 1, n, D, device="cuda", generator=g) + 2.0).bfloat16()


@gpu
def test_8_bit_cache():
    k, v = rows(T, 1)
    one, all_ = da.dash_cache_alloc(1, 1, T, D), da.dash_cache_alloc(1, H, T, D)
    assert all_[0].numel() > 1 << 32
    held = T - 200
    da.dash_cache_append(k, v, i32([0]), *one[:4], ksum=one[4], n=held)
    for x, y in zip(all_, one):
        x.view(torch.uint8)[:, -1:] = y.view(torch.uint8)
    # a tail appended in both: the last head's rows and summaries alike
    tail = [x[:, :, held:].contiguous() for x in (k, v)]
    wide = [torch.zeros(1, H, 200, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for x, y in zip(wide, tail):
        x[:, -1:] = y
    da.dash_cache_append(*tail, i32([held]), *one[:4], ksum=one[4])
    da.dash_cache_append(*wide, i32([held]), *all_[:4], ksum=all_[4])
    for x, y in zip(all_, one):
        assert same_bits(x[:, -1:], y)
    got, want = (da.dash_cache_read(*c[:4], 300, start=i32([held - 50])) for c in (all_, one))
    for x, y in zip(got, want):
        assert torch.equal(x[:, -1:], y) and bool((x[:, :-1] == 0).all())
    vmax = float(want[1].float().abs().max()) + 1.0
    q = k[:, :, 1000].contiguous()
    q_all = q.expand(1, H, D).contiguous()
    near(da.dash_decode_q8(q_all, *all_, i32([T - 3]), coarse_scale=CS)[0][:, -1:], da.dash_decode_q8(q, *one, i32([T - 3]), coarse_scale=CS)[0], vmax, 11)
    qt, kd, vd = k[:, :, 64:67].contiguous(), k[:, :, 128:131].contiguous(), v[:, :, :3].contiguous()
    wide = [x.expand(1, H, 3, D).contiguous() for x in (qt, kd, vd)]
    par, lens = i32([[-1, 0, 1]]), i32([T - 1])
    near(da.dash_decode_tree_q8(*wide, par, *all_, lens, coarse_scale=CS)[0][:, -1:],
         da.dash_decode_tree_q8(qt, kd, vd, par, *one, lens, coarse_scale=CS)[0], vmax, 8)


@gpu
def test_trees_over_a_bf16_cache():
    k, v = rows(T, 2)
    ks = da.dash_block_summary(k)
    k_all, v_all = (torch.zeros(1, H, T, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ks_all = torch.zeros(1, H, T // 64, D, device="cuda")
    for x, y in ((k_all, k), (v_all, v), (ks_all, ks)):
        x[:, -1:] = y
    qt, kd, vd = k[:, :, 64:67].contiguous(), k[:, :, 128:131].contiguous(), v[:, :, :3].contiguous()
    wide = [x.expand(1, H, 3, D).contiguous() for x in (qt, kd, vd)]
    par, lens = i32([[-1, 0, 1]]), i32([T - 1])
    near(da.dash_decode_tree(*wide, par, k_all, v_all, ks_all, lens, coarse_scale=CS)[0][:, -1:],
         da.dash_decode_tree(qt, kd, vd, par, k, v, ks, lens, coarse_scale=CS)[0], float(v.float().abs().max()), 8)
