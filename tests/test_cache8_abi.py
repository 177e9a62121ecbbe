"""Argument errors of the 8-bit cache and drafted-tree calls: all are found before any launch, so
they are checked here without a GPU."""
import ctypes

import pytest
import torch

f = ctypes.c_void_p
FAKE, OFF, BIG = f(1 << 20), f((1 << 20) + 8), 1 << 40


@pytest.fixture(scope="module")
def L():
    from sparse_hierarchical_attention_pool_b200 import build, dash_attn
    build.build()
    return dash_attn.lib()


def caller(fn, args):
    def call(**over):
        a = list(args)
        for i, v in over.items():
            a[int(i[1:])] = v
        return fn(*a)
    return call


def test_append_refusals(L):
    #        k_new v_new src n_new kv_len kc vc ks vs ksum | B Hkv rows n Tmax d block stream
    call = caller(L.dash_cache_append, [FAKE, FAKE, None, None] + [FAKE] * 5 + [None] + [1, 2, 8, 8, 128, 64, 64, None])
    for i in (0, 1, 4, 5, 6, 7, 8):
        assert call(**{f"a{i}": None}) == -1
    for i in (0, 1, 5, 6, 7, 8, 9):
        assert call(**{f"a{i}": OFF}) == -1
    assert call(a10=0) == -2 and call(a11=0) == -2
    assert call(a13=-1) == -2 and call(a13=9) == -2          # more tokens than rows
    assert call(a13=129, a12=200) == -2                       # more than the cache holds
    assert call(a12=-1, a13=0) == -2
    assert call(a14=100) == -2 and call(a14=0) == -2          # Tmax: whole blocks
    assert call(a14=(1 << 20) + 64) == -2
    assert call(a15=96) == -2 and call(a16=32) == -2
    assert call(a10=1 << 20, a11=64) == -2                    # 2^31 rows
    assert call(a13=0) == 0                                   # nothing to do


def test_read_refusals(L):
    #       kc vc ks vs start kv_len ko vo | B Hkv n Tmax d block stream
    call = caller(L.dash_cache_read, [FAKE] * 4 + [None, None, FAKE, FAKE] + [1, 2, 8, 128, 64, 64, None])
    for i in (0, 1, 2, 3, 6, 7):
        assert call(**{f"a{i}": None}) == -1 and call(**{f"a{i}": OFF}) == -1
    assert call(a10=-1) == -2 and call(a10=(1 << 20) + 1) == -2
    assert call(a11=65) == -2 and call(a12=32) == -2 and call(a13=128) == -2
    assert call(a10=0) == 0


def test_decode_q8_refusals(L):
    #       q kc vc ks vs ksum kv_len out | B Hq Hkv Tmax d block alpha cs ws bytes stream
    call = caller(L.dash_decode_q8, [FAKE] * 8 + [1, 4, 2, 128, 64, 64, 1.5, 1.0, FAKE, BIG, None])
    for i in range(8):
        assert call(**{f"a{i}": None}) == -1
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert call(**{f"a{i}": OFF}) == -1
    assert call(a14=1.0) == -1 and call(a14=float("nan")) == -1 and call(a15=float("inf")) == -1
    assert call(a9=3) == -2 and call(a11=100) == -2 and call(a12=80) == -2 and call(a13=32) == -2
    assert call(a9=66, a10=2) == -2                           # 33 heads per KV head
    assert call(a16=None) == -5 and call(a16=f((1 << 20) + 16)) == -5 and call(a17=64) == -5
    size = L.dash_decode_q8_workspace_size
    assert size(1, 4, 2, 128, 64, 64) > 0 and size(1, 4, 2, 100, 64, 64) == 0 and size(1, 33, 1, 128, 64, 64) == 0
    assert call(a17=size(1, 4, 2, 128, 64, 64) - 1) == -5


@pytest.mark.parametrize("q8", [False, True])
def test_tree_refusals(L, q8):
    #       q kd vd parent n_nodes kc vc [ks vs] ksum kv_len out | B Hq Hkv N Tmax d block alpha cs ws bytes stream
    n = 12 if q8 else 10
    fn = L.dash_decode_tree_q8 if q8 else L.dash_decode_tree
    call = caller(fn, [FAKE] * 4 + [None] + [FAKE] * (n - 5) + [1, 4, 2, 8, 128, 64, 64, 1.5, 1.0, FAKE, BIG, None])
    for i in range(n):
        if i != 4:
            assert call(**{f"a{i}": None}) == -1
        if i not in (3, 4, n - 2):
            assert call(**{f"a{i}": OFF}) == -1
    at = lambda k: f"a{n + k}"  # noqa: E731
    assert call(**{at(3): 0}) == -2 and call(**{at(3): 65}) == -2
    assert call(**{at(1): 3}) == -2 and call(**{at(1): 66}) == -2
    assert call(**{at(5): 96}) == -2 and call(**{at(6): 32}) == -2
    assert call(**{at(7): 1.0}) == -1 and call(**{at(8): float("nan")}) == -1
    assert call(**{at(9): None}) == -5 and call(**{at(10): 256}) == -5
    if q8:
        assert call(**{at(4): 100}) == -2                     # the 8-bit cache holds whole blocks
    size = L.dash_decode_tree_workspace_size
    assert size(1, 4, 2, 8, 100, 64, 64) > 0 and size(1, 4, 2, 65, 128, 64, 64) == 0
    assert size(8, 32, 8, 64, 98304, 128, 64) < 1 << 30
    assert call(**{at(10): size(1, 4, 2, 8, 128, 64, 64) - 1}) == -5


def test_binding_refuses_wrong_tensors_before_any_call():
    from sparse_hierarchical_attention_pool_b200 import dash_attn as da
    B, Hkv, T, d, n = 2, 1, 64, 64, 3
    x = torch.zeros(B, Hkv, n, d, dtype=torch.bfloat16)
    kc, vc, ks, vs, ksum = da.dash_cache_alloc(B, Hkv, T, d, device="cpu")
    lens = torch.zeros(B, dtype=torch.int32)
    with pytest.raises(ValueError):                           # CPU tensors: no CPU path
        da.dash_cache_append(x, x, lens, kc, vc, ks, vs, ksum=ksum)
    with pytest.raises(ValueError):
        da.dash_cache_append(x, x[:, :, :2], lens, kc, vc, ks, vs)
    with pytest.raises(ValueError):
        da.dash_cache_append(x, x, lens, kc[:1], vc, ks, vs)
    with pytest.raises(ValueError):
        da.dash_cache_append(x, x, lens, kc, vc, ks, vs, src=torch.zeros(1, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        da.dash_cache_read(kc, vc, ks, vs, 4)
    with pytest.raises(ValueError):
        da.dash_cache_alloc(1, 1, 100, 64, device="cpu")
    q = torch.zeros(B, 2, n, d, dtype=torch.bfloat16)
    par = torch.zeros(B, n, dtype=torch.int32)
    with pytest.raises(ValueError):
        da.dash_decode_tree(q, x, x, par[:, :2], x, x, ksum, lens)
    with pytest.raises(ValueError):
        da.dash_decode_tree(q, x, x[:, :, :1], par, x, x, ksum, lens)
    with pytest.raises(ValueError):
        da.dash_decode_q8(q[:, :, 0], kc, vc, ks, vs, ksum, lens, out=q)
