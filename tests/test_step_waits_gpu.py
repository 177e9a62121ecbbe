"""Steps whose CTAs take many short lists (the open block's and the draft's entries among every few): no wait
inside a kernel runs to its limit of two seconds, not even the one for the last copies."""
import pytest
import torch

from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import filled, i32
from test_tree_gpu import CS, drafts

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("op", ["decode_q8", "tree", "tree_q8"])
@pytest.mark.parametrize("B", [3, 400])
def test_no_wait_runs_out(B, op):
    Hq, Hkv, T, d, N = 4, 2, 192, 64, 3
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=261)
    q, kd, vd = (x.cuda() for x in drafts(B, Hq, Hkv, N, d, 262))
    c, lens, par = filled(B, Hkv, T, d, k, v), i32([1 + 37 * b % 192 for b in range(B)]), i32([[-1, 0, 0]] * B)
    kc, vc, q1 = k.cuda(), v.cuda(), q4[:, :, 3].contiguous().cuda()
    ksum = da.dash_block_summary(kc)
    call = {"decode_q8": lambda: da.dash_decode_q8(q1, *c, lens, coarse_scale=CS),
            "tree": lambda: da.dash_decode_tree(q, kd, vd, par, kc, vc, ksum, lens, coarse_scale=CS),
            "tree_q8": lambda: da.dash_decode_tree_q8(q, kd, vd, par, *c, lens, coarse_scale=CS)}[op]
    call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    _, ws = call()
    end.record()
    torch.cuda.synchronize()
    assert da.dash_get_device_status(ws) == 0
    assert start.elapsed_time(end) < 500.0
