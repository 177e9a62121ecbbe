"""Steps called by host threads at once (the binding lets go of the interpreter lock), over caches of
different lengths: no call fails, and each gives what it gives alone."""
import ctypes
import threading

import pytest
import torch

from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs
from test_cache8_gpu import filled, i32

gpu = pytest.mark.gpu
CS = 0.05


def make(op, T, Hq, Hkv, d, seed):
    """A call without arguments, its workspace and output its own."""
    _, (q4, k, v) = inputs.make("16k", B=1, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=4, seed=seed)
    kc, vc, lens = k.cuda(), v.cuda(), i32([T - 3])
    q = q4[:, :, 5].contiguous().cuda()
    if op == "decode":
        ksum = da.dash_block_summary(kc)
        out, ws = torch.empty_like(q), da.alloc_workspace(da.decode_workspace_size(1, Hq, Hkv, T, d))
        return out, lambda: da.dash_decode(q, kc, vc, ksum, lens, out=out, coarse_scale=CS, workspace=ws)
    c = filled(1, Hkv, T, d, k, v)
    if op == "decode_q8":
        out, ws = torch.empty_like(q), da.alloc_workspace(da.decode_q8_workspace_size(1, Hq, Hkv, T, d))
        return out, lambda: da.dash_decode_q8(q, *c, lens, out=out, coarse_scale=CS, workspace=ws)
    qd, kd, vd = (x[:, :, :4].contiguous().cuda() for x in (q4, k, v))
    par = i32([[-1, 0, 1, 0]])
    out, ws = torch.empty_like(qd), da.alloc_workspace(da.decode_tree_workspace_size(1, Hq, Hkv, 4, T, d))
    return out, lambda: da.dash_decode_tree_q8(qd, kd, vd, par, *c, lens, out=out, coarse_scale=CS, workspace=ws)


def bare(call):
    """The library function that `call` reaches, and its arguments without the stream."""
    real, seen = da.lib(), []

    class Recorder:
        def __getattr__(self, name):
            fn = getattr(real, name)
            return lambda *a: (seen.append((fn, a)), fn(*a))[1]

    da._lib = Recorder()
    try:
        call()
    finally:
        da._lib = real
    return seen[-1][0], seen[-1][1][:-1]


def race(calls, steps=4000):
    """Every call alone, then all of them from threads of their own, without the binding's own time between."""
    alone, status, go = [], [[] for _ in calls], threading.Barrier(len(calls))
    for out, call in calls:
        call()
        torch.cuda.synchronize()
        alone.append(out.clone())

    def work(fn, args, stream, status):
        go.wait()
        for _ in range(steps):
            status.append(fn(*args, stream))

    streams = [torch.cuda.Stream() for _ in calls]
    threads = [threading.Thread(target=work, args=(*bare(c[1]), ctypes.c_void_p(s.cuda_stream), st))
               for c, s, st in zip(calls, streams, status)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for st, (out, _), want in zip(status, calls, alone):
        assert st == [0] * steps, f"{steps - st.count(0)} of {steps} calls failed"
        assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("op", ["decode", "decode_q8", "tree_q8"])
def test_threads_with_caches_of_different_lengths(op):
    """Four threads a length: what a step asks of a kernel's shared memory follows from the cache's length."""
    race([make(op, T, 2, 1, 64, i) for i, T in enumerate((64, 4096) * 4)])


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_threads_with_different_numbers_of_heads(d):
    """More than 8 heads per KV head: the attention's shared memory grows with their number."""
    race([make("decode", 128, Hq, 1, d, i) for i, Hq in enumerate((9, 32) * 4)])
