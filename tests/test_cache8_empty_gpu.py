"""Appending no tokens, in each way that a caller can say so, is no error and changes nothing."""
import pytest
import torch

from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from test_cache8_gpu import i32, junk_cache, rows, same_bits

gpu = pytest.mark.gpu


@gpu
def test_appending_no_tokens():
    B, Hkv, T, d = 2, 2, 128, 64
    c = junk_cache(B, Hkv, T, d)
    before = [t.clone() for t in c]
    none = torch.empty(B, Hkv, 0, d, dtype=torch.bfloat16, device="cuda")
    some = rows(B, Hkv, 3, d, 1).cuda()
    lens, no_src = i32([5, 63]), torch.empty(B, 0, dtype=torch.int32, device="cuda")
    for x, kw in ((none, {}), (some, {"n": 0}), (some, {"src": no_src}), (none, {"src": no_src}), (some, {"n_new": i32([0, 0])})):
        da.dash_cache_append(x, x, lens, *c[:4], ksum=c[4], **kw)
        for a, b in zip(c, before):
            assert same_bits(a, b)
    with pytest.raises(ValueError):                                  # the other arguments are still looked at
        da.dash_cache_append(none, none, lens.cpu(), *c[:4])
    with pytest.raises(ValueError):
        da.dash_cache_append(none, none, lens, c[0], c[1], c[2][:, :, :64], c[3])
