"""Appending no tokens, in each way that a caller can say so, is no error and changes nothing; what is no tensor is
a ValueError like any other wrong argument."""
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
    for x, kw in ((none, {}), (some, {"n": 0}), (some, {"src": no_src}), (none, {"src": no_src}), (some, {"n_new": i32([0, 0])}),
                  (none, {"src": i32([[0], [0]])})):                 # no row 0: the sequences are left as they were
        da.dash_cache_append(x, x, lens, *c[:4], ksum=c[4], **kw)
        for a, b in zip(c, before):
            assert same_bits(a, b)
    with pytest.raises(ValueError):                                  # the other arguments are still looked at
        da.dash_cache_append(none, none, lens.cpu(), *c[:4])
    with pytest.raises(ValueError):
        da.dash_cache_append(none, none, lens, c[0], c[1], c[2][:, :, :64], c[3])


@gpu
def test_what_is_no_tensor_and_summaries_without_rows_are_refused():
    B, Hkv, T, d = 1, 1, 64, 64
    c, x, lens = junk_cache(B, Hkv, T, d), rows(B, Hkv, 3, d, 1).cuda(), i32([0])
    q, par = x[:, :, 0].contiguous(), i32([[-1, 0, 1]])
    for bad in (None, 5, lens.cpu().numpy(), [0]):
        with pytest.raises(ValueError):
            da.dash_cache_append(x, x, bad, *c[:4])
        with pytest.raises(ValueError):
            da.dash_cache_append(x, bad, lens, *c[:4])
        with pytest.raises(ValueError):
            da.dash_decode_q8(q, *c[:4], bad, lens)
        with pytest.raises(ValueError):
            da.dash_decode_tree_q8(x, x, x, par, *c, bad)
    short = torch.zeros(B, Hkv, 40, d, dtype=torch.bfloat16, device="cuda")      # no whole block: one summary row
    for n, ok in ((1, True), (0, False)):
        ksum = torch.zeros(B, Hkv, n, d, device="cuda")
        if ok:
            out, _ = da.dash_decode_tree(x, x, x, par, short, short, ksum, lens)
            assert bool(torch.isfinite(out).all())
        else:
            with pytest.raises(ValueError):
                da.dash_decode_tree(x, x, x, par, short, short, ksum, lens)
