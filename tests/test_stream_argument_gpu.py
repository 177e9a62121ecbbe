"""The 8-bit cache's and the trees' calls with a stream argument: what a call allocates for itself belongs to
the stream that its kernels run on, not to the current one."""
import pytest
import torch

from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import filled, i32

gpu = pytest.mark.gpu


def problem(T=512, Hq=4, Hkv=2, d=64, N=4):
    _, (q4, k, v) = inputs.make("16k", B=2, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=3, seed=61)
    qd, kd, vd = (x[:, :, :N].contiguous().cuda() for x in (q4, k, v))
    c, lens, par = filled(2, Hkv, T, d, k, v), i32([T - 9, 100]), i32([[-1, 0, 1, 0]] * 2)
    kc, vc = k.cuda(), v.cuda()
    ksum = da.dash_block_summary(kc)
    q = q4[:, :, 7].contiguous().cuda()
    return {
        "read": lambda **kw: da.dash_cache_read(*c[:4], 300, start=i32([5, 60]), **kw),
        "decode_q8": lambda **kw: da.dash_decode_q8(q, *c, lens, coarse_scale=0.05, **kw),
        "tree": lambda **kw: da.dash_decode_tree(qd, kd, vd, par, kc, vc, ksum, lens, coarse_scale=0.05, **kw),
        "tree_q8": lambda **kw: da.dash_decode_tree_q8(qd, kd, vd, par, *c, lens, coarse_scale=0.05, **kw),
    }


@gpu
@pytest.mark.parametrize("op", ["read", "decode_q8", "tree", "tree_q8"])
def test_a_calls_own_tensors_belong_to_its_stream(op):
    call, side = problem()[op], torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    got = call(stream=side)
    torch.cuda.synchronize()
    if op == "read":
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        assert torch.equal(got[0], want[0])
    where = [(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in got]
    del got
    # blocks that the allocator hands to the current stream now are none of the side stream's
    fresh = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in where for _ in range(2)]
    for f in fresh:
        for p, n in where:
            assert f.data_ptr() + f.numel() <= p or p + n <= f.data_ptr()


@gpu
@pytest.mark.parametrize("op", ["read", "decode_q8", "tree", "tree_q8"])
def test_pending_work_on_the_current_stream_does_not_reach_a_calls_tensors(op):
    """Memory that the current stream is still to write is freed, then the call runs on another stream."""
    call, side = problem()[op], torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    late = [torch.empty_like(t.view(torch.uint8)) for t in want]
    torch.cuda._sleep(20_000_000)
    for t in late:
        t.fill_(77)
    del late, t
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in list(zip(got, want))[:2 if op == "read" else 1]:
        assert torch.equal(a, b)
    if op != "read":
        assert da.dash_get_device_status(got[1]) == 0
