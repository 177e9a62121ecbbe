"""The 8-bit KV cache on the GPU: codes, scales and summaries of dash_cache_append against a
64-bit rounding on the e4m3 grid, dash_cache_read, and dash_decode_q8 against the fp64 oracle on
the values that the cache holds."""
import math

import numpy as np
import pytest
import torch

import oracle
from sparse_hierarchical_attention_pool_b200 import dash_attn as da
from sparse_hierarchical_attention_pool_b200 import inputs

gpu = pytest.mark.gpu


def reference(x):
    """Values (fp64) and scale bytes of rows x, rounded on the e4m3 grid in 64 bits."""
    x = x.double()
    bad = ~torch.isfinite(x).all(-1)
    mag = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    e = torch.full_like(mag, -118)
    for cand in range(121, -119, -1):
        e = torch.where(mag <= 448.0 * 2.0 ** cand, torch.full_like(e, max(cand, -118)), e)
    y = x * torch.exp2(-e).unsqueeze(-1)
    y = torch.where((e == 120).unsqueeze(-1), y.clamp(-240.0, 240.0), y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    v = torch.round(y / step) * step * torch.exp2(e).unsqueeze(-1)
    v[bad] = math.nan
    return v, torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def held(code, scale):
    """fp64 values that codes and scale bytes stand for."""
    f = torch.exp2(scale.double() - 127)
    f[scale == 255] = math.nan
    return code.double() * f.unsqueeze(-1)


def rows(B, Hkv, n, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, Hkv, n, d, generator=g) * torch.exp(2 * torch.randn(B, Hkv, n, 1, generator=g))
    return x.bfloat16()


def junk_cache(B, Hkv, T, d, seed=3):
    """A cache whose every byte is arbitrary (NaN codes and scales among them)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    return (r(B, Hkv, T, d).view(torch.float8_e4m3fn), r(B, Hkv, T, d).view(torch.float8_e4m3fn),
            r(B, Hkv, T), r(B, Hkv, T), torch.full((B, Hkv, T // 64, d), 7.0, device="cuda"))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def equal_values(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,T,lens", [(1, 64, [0, 63]), (1, 128, [63, 64]), (2, 128, [63, 126]), (64, 192, [0, 1]),
                                      (66, 256, [63, 64]), (130, 256, [5, 126])])
def test_append_codes_scales_and_summaries(n, T, lens, d):
    B, Hkv = 2, 3
    k, v = rows(B, Hkv, n, d, 1), rows(B, Hkv, n, d, 2)
    kc, vc, ks, vs, ksum = junk_cache(B, Hkv, T, d)
    # what is held before the call must be finite where a summary takes it
    kc0, vc0 = rows(B, Hkv, T, d, 4), rows(B, Hkv, T, d, 5)
    if max(lens) > 0:
        da.dash_cache_append(kc0.cuda(), vc0.cuda(), i32([0] * B), kc, vc, ks, vs, n=max(lens), n_new=i32(lens))
    before = [t.clone() for t in (kc, vc, ks, vs, ksum)]
    da.dash_cache_append(k.cuda(), v.cuda(), i32(lens), kc, vc, ks, vs, ksum=ksum)
    for new, code, scale, old_code, old_scale in ((k, kc, ks, before[0], before[2]), (v, vc, vs, before[1], before[3])):
        want, want_scale = reference(new)
        for b, L in enumerate(lens):
            got = held(code[b, :, L:L + n].float().cpu(), scale[b, :, L:L + n].cpu())
            assert torch.equal(scale[b, :, L:L + n].cpu(), want_scale[b])
            assert equal_values(got, want[b])
            for lo, hi in ((0, L), (L + n, T)):                       # every other row is as it was
                assert same_bits(code[b, :, lo:hi], old_code[b, :, lo:hi])
                assert torch.equal(scale[b, :, lo:hi], old_scale[b, :, lo:hi])
    allk = held(kc.float().cpu(), ks.cpu())
    for b, L in enumerate(lens):
        for j in range(T // 64):
            if L // 64 <= j < (L + n) // 64:
                blk = allk[b, :, 64 * j:64 * j + 64]
                # 64 fp32 additions: off by at most 64 2^-24 of the sum of magnitudes
                tol = 2.0 ** -18 * blk.abs().sum(1) / 64
                assert bool(((ksum[b, :, j].cpu().double() - blk.mean(1)).abs() <= tol).all())
            else:
                assert bool((ksum[b, :, j] == 7.0).all())


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_special_rows(d):
    """Zeros, ties, subnormals, the largest numbers, and rows that are not finite."""
    big = torch.finfo(torch.bfloat16).max
    r = torch.zeros(12, d, dtype=torch.float64)
    r[1] = -0.0
    r[2, 0], r[2, 1:] = 448.0, torch.tensor([17.0, 18.0, 19.0, 21.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10]).repeat(d)[:d - 1]
    r[3, 0], r[3, 1] = 449.0 + 1.0, 1.0                            # 450 -> 448 or 452 in bf16: the scale steps up
    r[4] = 2.0 ** -133                                              # the least bf16 subnormal
    r[5], r[5, 1] = big, -big / 3
    r[6] = 2.0 ** -126
    r[7, 3] = math.nan
    r[8, d - 1] = math.inf
    r[9, 0] = -math.inf
    r[10] = math.nan
    r[11, 0], r[11, 1] = 1.0, 2.0 ** -30
    x = r.bfloat16().view(1, 1, 12, d)
    kc, vc, ks, vs, ksum = junk_cache(1, 1, 64, d)
    da.dash_cache_append(x.cuda(), x.cuda(), i32([0]), kc, vc, ks, vs, ksum=ksum)
    want, scale = reference(x)
    for code, s in ((kc, ks), (vc, vs)):
        assert torch.equal(s[:, :, :12].cpu(), scale)
        assert equal_values(held(code[:, :, :12].float().cpu(), s[:, :, :12].cpu()), want)
    k, v = da.dash_cache_read(kc, vc, ks, vs, 12)
    assert equal_values(k.double().cpu(), want) and equal_values(v.double().cpu(), want)     # exact in bf16
    assert torch.isfinite(kc[:, :, :12].float()).all()              # codes are never NaN


@gpu
def test_append_one_by_one_equals_at_once():
    B, Hkv, n, d, T = 2, 2, 150, 128, 192
    k, v = rows(B, Hkv, n, d, 6).cuda(), rows(B, Hkv, n, d, 7).cuda()
    a, b = junk_cache(B, Hkv, T, d), junk_cache(B, Hkv, T, d)
    da.dash_cache_append(k, v, i32([3, 20]), *a[:4], ksum=a[4])
    for i in range(n):
        da.dash_cache_append(k[:, :, i:i + 1].contiguous(), v[:, :, i:i + 1].contiguous(), i32([3 + i, 20 + i]), *b[:4], ksum=b[4])
    for x, y in zip(a, b):
        assert same_bits(x, y)
    # rejected tokens are written over: the summaries follow what is held
    da.dash_cache_append(v, k, i32([60, 60]), *b[:4], ksum=b[4], n=30)
    da.dash_cache_append(k, v, i32([60, 60]), *b[:4], ksum=b[4], src=torch.arange(57, 87, device="cuda", dtype=torch.int32).repeat(2, 1))
    assert same_bits(a[0][0], b[0][0]) and same_bits(a[4][0], b[4][0])   # NaN where junk rows were held before


@gpu
def test_append_rows_by_index_and_counts():
    B, Hkv, rws, d, T = 5, 2, 7, 64, 128
    k, v = rows(B, Hkv, rws, d, 8), rows(B, Hkv, rws, d, 9)
    cache = junk_cache(B, Hkv, T, d)
    before = [t.clone() for t in cache]
    src = i32([[0, 2, 2, 6], [6, 5, 4, 3], [1, 9, 1, 1], [1, 1, 9, 1], [0, 1, 2, 3]])
    n_new = i32([4, 0, 3, 2, 4])
    lens = [62, 10, 62, 62, 125]                                     # sequence 2: index 9; sequence 4: no room
    da.dash_cache_append(k.cuda(), v.cuda(), i32(lens), *cache[:4], ksum=cache[4], src=src, n_new=n_new)
    for b, m in ((0, 4), (1, 0), (2, 0), (3, 2), (4, 0)):
        L, idx = lens[b], src[b, :m].cpu().long()
        want, scale = reference(v[b][:, idx])
        assert equal_values(held(cache[1][b, :, L:L + m].float().cpu(), cache[3][b, :, L:L + m].cpu()), want)
        for x, y in zip(cache[:4], before[:4]):
            assert same_bits(x[b, :, :L], y[b, :, :L]) and same_bits(x[b, :, L + m:], y[b, :, L + m:])
    bad = junk_cache(B, Hkv, T, d)
    da.dash_cache_append(k.cuda(), v.cuda(), i32([-1, 129, 122, 0, 0]), *bad[:4], ksum=bad[4], n_new=i32([1, 0, 7, -1, 8]), n=7)
    ref = junk_cache(B, Hkv, T, d)
    for x, y in zip(bad, ref):
        assert same_bits(x, y)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_read_ranges(d):
    B, Hkv, T = 3, 2, 192
    k, v = rows(B, Hkv, T, d, 10), rows(B, Hkv, T, d, 11)
    c = junk_cache(B, Hkv, T, d)[:4]
    da.dash_cache_append(k.cuda(), v.cuda(), i32([0] * B), *c)
    want = [reference(k)[0].float(), reference(v)[0].float()]
    for n, start, lens in ((T, None, None), (1, [0, 191, 63], None), (33, [-5, 180, 100], [192, 192, 110]), (70, [0, 0, 0], [0, 1, 300]), (0, None, None)):
        got = da.dash_cache_read(*c, n, start=None if start is None else i32(start), kv_len=None if lens is None else i32(lens))
        for g, w in zip(got, want):
            assert g.shape == (B, Hkv, n, d)
            for b in range(B):
                for i in range(n):
                    t = (start[b] if start else 0) + i
                    ok = 0 <= t < min(T, lens[b] if lens else T)
                    assert torch.equal(g[b, :, i].float().cpu(), w[b, :, t] if ok else torch.zeros(Hkv, d))


# ---------------------------------------------------------------- decode over the cache

def weight_error(alpha, w_bits):
    """Bound on the relative error of a softmax weight: its rounding to w_bits significant bits
    (2^-w_bits), the fp32 logit and prior (2^-10 covers 128 2^-24 of magnitudes up to 700 and the
    prior's slope), and for alpha > 2 the prior's root at the border, (4 2^-15)^(1 / (alpha - 1))."""
    edge = (4 * 2.0 ** -15) ** (1 / (alpha - 1)) if alpha > 2 else 0.0
    return 2.0 ** -w_bits + 2.0 ** -10 + edge


def close(got, ref, vmax, alpha, w_bits, what=""):
    """bf16 output: half a step (2^-8 of the value), and weights off by a relative rho each move a
    convex combination of values by at most 2 rho max|v|."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.isfinite(got).all(), what
    tol = 2.0 ** -8 * np.abs(ref) + 2 * weight_error(alpha, w_bits) * vmax
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"{what}: {(err / tol).max():.2f} x its tolerance"


def filled(B, Hkv, T, d, k, v):
    c = junk_cache(B, Hkv, T, d)
    da.dash_cache_append(k.cuda(), v.cuda(), i32([0] * B), *c[:4], ksum=c[4], n=T)
    return c


@gpu
@pytest.mark.parametrize("Hq,Hkv,d,alpha", [(1, 1, 64, 1.5), (4, 1, 128, 1.5), (6, 2, 128, 2.0), (8, 1, 64, 1.25), (7, 1, 128, 3.0),
                                            (12, 1, 128, 1.5), (9, 1, 64, 2.0), (22, 2, 64, 1.5), (32, 1, 128, 1.5)])
def test_decode_q8_against_oracle(Hq, Hkv, d, alpha):
    B, T = 6, 640
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=4, seed=21 + Hq)
    c = filled(B, Hkv, T, d, k, v)
    kh, vh = da.dash_cache_read(*c[:4], T)
    lens = [1, 63, 64, 65, 449, 640]
    q = torch.stack([q4[b, :, lens[b] - 1] for b in range(B)]).contiguous()
    out, ws = da.dash_decode_q8(q.cuda(), *c, i32(lens), alpha=alpha, coarse_scale=0.05)
    assert da.dash_get_device_status(ws) == 0
    rws = [(b, h, lens[b] - 1) for b in range(B) for h in range(Hq)]
    ref, _, _ = oracle.forward_rows(q.reshape(-1, d), kh.cpu(), vh.cpu(), rws, Hq, 64, alpha, 0.05)
    close(out.float().cpu().reshape(-1, d), ref, float(vh.float().abs().max()), alpha, 11, f"G={Hq // Hkv} d={d}")


@gpu
def test_decode_q8_junk_behind_the_sequence_and_bad_lengths():
    B, Hq, Hkv, T, d = 4, 8, 2, 192, 128
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=5)
    lens = [70, 1, 0, 193]
    c = junk_cache(B, Hkv, T, d)                                     # every byte behind the sequences is arbitrary
    da.dash_cache_append(k.cuda(), v.cuda(), i32([0] * B), *c[:4], ksum=c[4], n=T, n_new=i32([70, 1, 0, 0]))
    q = q4[:, :, 0].contiguous()
    out, _ = da.dash_decode_q8(q.cuda(), *c, i32(lens), coarse_scale=0.05)
    kh, vh = da.dash_cache_read(*c[:4], T, kv_len=i32([70, 1, 0, 0]))
    rws = [(b, h, lens[b] - 1) for b in range(2) for h in range(Hq)]
    ref, _, _ = oracle.forward_rows(q[:2].reshape(-1, d), kh.cpu(), vh.cpu(), rws, Hq, 64, 1.5, 0.05)
    close(out[:2].float().cpu().reshape(-1, d), ref, float(vh.float().abs().max()), 1.5, 11)
    assert bool((out[2:] == 0).all())


@gpu
def test_decode_q8_value_scales_that_differ_widely():
    """Values whose scales span 2^80: each head's output keeps the relative accuracy of its own values."""
    B, Hq, Hkv, T, d = 1, 4, 1, 256, 64
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=4, seed=8)
    for p, mul in ((0, 2.0 ** -40), (1, 1.0), (2, 2.0 ** 40), (3, 2.0 ** -70)):
        _, (_, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=4, seed=8)
        v = (v.float() * mul).bfloat16()
        if p == 1:
            v[:, :, 64:128] = (v[:, :, 64:128].float() * 2.0 ** -30).bfloat16()
        c = filled(B, Hkv, T, d, k, v)
        kh, vh = da.dash_cache_read(*c[:4], T)
        q = q4[:, :, 255].contiguous()
        out, _ = da.dash_decode_q8(q.cuda(), *c, i32([256]), coarse_scale=0.05)
        ref, _, _ = oracle.forward_rows(q.reshape(-1, d), kh.cpu(), vh.cpu(), [(0, h, 255) for h in range(Hq)], Hq, 64, 1.5, 0.05)
        close(out.float().cpu().reshape(-1, d), ref, float(vh.float().abs().max()), 1.5, 11, f"scale {mul}")


@gpu
def test_decode_q8_nan_row_stays_with_its_readers():
    """A value row that is NaN reaches the heads that attend its block, and no other head or sequence."""
    B, Hq, Hkv, T, d = 2, 2, 1, 320, 64
    g = torch.Generator().manual_seed(3)
    k, v = torch.zeros(B, Hkv, T, d), torch.randn(B, Hkv, T, d, generator=g)
    k[:, :, 0:64, 0] = 4.0                                           # block 0 points along dim 0, block 1 along dim 1
    k[:, :, 64:128, 1] = 4.0
    q = torch.zeros(B, Hq, d)
    q[:, 0, 0], q[:, 1, 1] = 8.0, 8.0                                # head 0 selects block 0 alone, head 1 block 1
    v[0, 0, 5, 7] = math.nan
    c = filled(B, Hkv, T, d, k.bfloat16(), v.bfloat16())
    out, _ = da.dash_decode_q8(q.bfloat16().cuda(), *c, i32([320, 320]), coarse_scale=1.0)
    assert bool(out[0, 0].isnan().all())
    assert bool(torch.isfinite(out[0, 1]).all()) and bool(torch.isfinite(out[1]).all())


@gpu
def test_decode_q8_many_sequences_split_over_ctas():
    """Lists long enough that groups are split over CTAs and merged, against decode on the held values."""
    B, Hq, Hkv, T, d = 3, 16, 2, 16384, 128
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=8, seed=31)
    c = filled(B, Hkv, T, d, k, v)
    lens = [16384, 9001, 15]
    kh, vh = da.dash_cache_read(*c[:4], T)
    q = q4[:, :, 100].contiguous()
    out, _ = da.dash_decode_q8(q.cuda(), *c, i32(lens), coarse_scale=0.05)
    rws = [(b, h, lens[b] - 1) for b in range(B) for h in range(Hq)]
    ref, _, _ = oracle.forward_rows(q.reshape(-1, d), kh.cpu(), vh.cpu(), rws, Hq, 64, 1.5, 0.05)
    close(out.float().cpu().reshape(-1, d), ref, float(vh.float().abs().max()), 1.5, 11)
    again, _ = da.dash_decode_q8(q.cuda(), *c, i32(lens), coarse_scale=0.05)
    assert torch.equal(out, again)                                   # the same every time


@gpu
def test_decode_q8_more_groups_than_a_merge_adds_up():
    """From 1024 lists on, the merge looks its pieces up in what the attention left: sampled sequences,
    empty ones among them, against the oracle."""
    B, Hq, Hkv, T, d = 520, 4, 2, 128, 64
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=2, seed=41)
    c = filled(B, Hkv, T, d, k, v)
    lens = [(37 * b) % 129 for b in range(B)]
    kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
    q = q4[:, :, 5].contiguous()
    out, ws = da.dash_decode_q8(q.cuda(), *c, i32(lens), coarse_scale=0.05)
    assert da.dash_get_device_status(ws) == 0
    out = out.float().cpu()
    some = [0, 1, 2, 7, 100, 255, 256, 511, 512, 518, 519] + [b for b in range(B) if lens[b] in (0, 64, 65, 128)][:8]
    for b in some:
        if lens[b] == 0:
            assert bool((out[b] == 0).all())
            continue
        ref, _, _ = oracle.forward_rows(q[b], kh[b:b + 1], vh[b:b + 1], [(0, h, lens[b] - 1) for h in range(Hq)], Hq, 64, 1.5, 0.05)
        close(out[b], ref, float(vh[b].float().abs().max()), 1.5, 11, f"sequence {b}")


@gpu
def test_decode_q8_rows_longer_than_the_shared_buffer():
    """More blocks than a warp keeps in shared memory (4096): the rest of a row is read from memory."""
    B, Hq, Hkv, T, d = 1, 2, 1, 262144 + 640, 64
    _, (q4, k, v) = inputs.make("16k", B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=8, seed=43)
    c = filled(B, Hkv, T, d, k, v)
    kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
    for L in (T, 262145 + 40):
        q = q4[:, :, L - 1].contiguous()
        out, _ = da.dash_decode_q8(q.cuda(), *c, i32([L]), coarse_scale=0.05)
        ref, _, _ = oracle.forward_rows(q.reshape(-1, d), kh, vh, [(0, h, L - 1) for h in range(Hq)], Hq, 64, 1.5, 0.05)
        close(out.float().cpu().reshape(-1, d), ref, float(vh.float().abs().max()), 1.5, 11, f"L={L}")


@gpu
def test_decode_q8_two_calls_at_once_and_any_workspace():
    """Calls on two streams with workspaces of their own, whatever the workspaces held, give what one
    call alone gives, bit for bit."""
    Hq, Hkv, d = 16, 2, 128
    calls = []
    for T, seed in ((8192, 61), (4096, 62)):
        _, (q4, k, v) = inputs.make("16k", B=2, Hq=Hq, Hkv=Hkv, T=T, d=d, n_topics=8, seed=seed)
        c = filled(2, Hkv, T, d, k, v)
        q, lens = q4[:, :, 9].contiguous().cuda(), i32([T, T // 2 + 3])
        alone, ws = da.dash_decode_q8(q, *c, lens, coarse_scale=0.05)
        calls.append((q, c, lens, alone, torch.full_like(ws, 255), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for q, c, lens, _, ws, s in calls:
            with torch.cuda.stream(s):
                outs.append(da.dash_decode_q8(q, *c, lens, coarse_scale=0.05, workspace=ws)[0])
        torch.cuda.synchronize()
        for o, call in zip(outs, calls):
            assert torch.equal(o, call[3])


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_and_read_at_the_largest_bf16_numbers(d):
    """Rows whose magnitudes end at bf16's largest: held as 240 2^120 at most, and read back finite."""
    x = torch.zeros(1, 1, 64, d)
    top = float(torch.finfo(torch.bfloat16).max)
    for i in range(64):
        x[0, 0, i, i % d] = (-1) ** i * top * 2.0 ** (-i / 4)
        x[0, 0, i, (i + 1) % d] = top / 3 if i % 2 else 2.0 ** -130
    x = x.bfloat16()
    c = junk_cache(1, 1, 64, d)
    da.dash_cache_append(x.cuda(), (-x).cuda(), i32([0]), *c[:4], ksum=c[4], n=64)
    want, scale = reference(x)
    assert torch.equal(c[2].cpu(), scale)
    k, v = da.dash_cache_read(*c[:4], 64)
    assert torch.equal(k.double().cpu(), want) and torch.equal(v.double().cpu(), -want)
    assert bool(torch.isfinite(k).all()) and float(k.abs().max()) <= 240 * 2.0 ** 120


@gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_decode_q8_query_or_key_that_is_no_number(bad):
    """A head whose query holds one is NaN; a key that holds one is NaN to the heads that attend its block.
    The other heads are right."""
    B, Hq, Hkv, T, d = 1, 4, 1, 256, 64
    g = torch.Generator().manual_seed(5)
    k, v = torch.zeros(B, Hkv, T, d), torch.randn(B, Hkv, T, d, generator=g)
    for j in range(3):
        k[:, :, 64 * j:64 * j + 64, j] = 4.0                         # block j points along dim j
    q = torch.zeros(B, Hq, d)
    for h in range(3):
        q[:, h, h] = 8.0                                             # head h selects block h alone
    q[:, 3, 0], q[:, 3, 9] = 8.0, bad
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    c = filled(B, Hkv, T, d, k, v)
    kh, vh = (x.cpu() for x in da.dash_cache_read(*c[:4], T))
    ref, _, _ = oracle.forward_rows(q[0], kh, vh, [(0, h, T - 1) for h in range(3)], Hq, 64, 1.5, 1.0)
    out, _ = da.dash_decode_q8(q.cuda(), *c, i32([T]), coarse_scale=1.0)
    assert bool(out[0, 3].isnan().all())
    close(out[0, :3].float().cpu(), ref, float(vh.float().abs().max()), 1.5, 11)
    k[0, 0, 70, 5] = bad                                             # in block 1, whose summary stays as it was
    da.dash_cache_append(k[:, :, 70:71].contiguous().cuda(), v[:, :, 70:71].contiguous().cuda(), i32([70]), *c[:4])
    out, _ = da.dash_decode_q8(q.cuda(), *c, i32([T]), coarse_scale=1.0)
    assert bool(out[0, 1].isnan().all())
    close(out[0, [0, 2]].float().cpu(), ref[[0, 2]], float(vh.float().abs().max()), 1.5, 11)
