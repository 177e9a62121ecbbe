// decode_q8.cu -- split-KV attention of a decode step over the 8-bit KV cache.
//
// The arithmetic of decode_tc.cu on the values that the cache holds (code 2^(s - 127),
// cache8.cuh), with its even split over the concatenated block lists.  What differs:
//
// Warps of a CTA share the ring that one producer lane fills and nothing else: each keeps a
// softmax state of its own and leaves it as a partial at the end of a group, and a second kernel
// merges a head's partials.  (Merging the warps in shared memory and the CTAs by a ticket cost
// each end of a group 8 us, of which a fifth of the CTAs has two.)  Bound by HBM where lists are long:
// at 96K, 8 sequences of 32 / 8 heads, the listed blocks' 369 MB take 65 us, 5.7 TB/s (the copies without
// the arithmetic took as long); at 16K, one sequence, 6 of a step's 22 us, which are latencies.
//
// Sums are fp32 (the e4m3 products of mma.sync too: 2^-25 of the sum of magnitudes at worst over
// random inputs), and the power-of-two scales stay outside the products:
//   K: the codes as they are, against q in two e4m3 parts: q' = q 2^-e_q = hi + lo / 16 with the
//      head's largest magnitude in [2^7, 2^8).  hi holds the leading 4 of q's 8 significant bits
//      and lo the other 4, so q' is exact over the 14 binades of e4m3's normal numbers, and what
//      lies deeper is off by at most 2^-14, 2^-21 of the largest.
//      logit = (hi . code + (lo . code) / 16) 2^(s_k - 127) 2^e_q / sqrt(d).
//   V: the codes as f16, in which every e4m3 number is exact.  The weight that multiplies a key's codes is w = 2^(l + s_v - 127 - mB), l the logit (log2)
//      and mB the running maximum of l + s_v - 127 over the keys so far, so that w lies in
//      (0, 2^kWBits] whatever the scales are and its rounding to f16 (11 bits) is relative to
//      the largest contribution.  The softmax's sum has its own maximum mA over l.
// The sum takes the unrounded weights: w's rounding is 2^-12, far below bf16 output's 2^-9.
//
// Fragments straight from the codes.  A consumer computes S^T = K Q^T (m16n8k32) and
// O^T += V^T W^T (m16n8k16; 32 keys are two M tiles, the group's <= 8 heads the N columns), and the order of
// dims inside a contraction, of output rows, and of the keys of a unit is free, so a lane takes
// 16 consecutive bytes per shared-memory load:
//   K: slots 4 t4 + 0 .. 3 and 16 + 4 t4 + 0 .. 3 of a 32-dim step i are dims 16 t4 + 8 i + 0 .. 7
//      of the 64-dim half;
//   V: lane row g4 owns dims 16 g4 .. 16 g4 + 15 (d = 64: 8 g4 .. + 7): M tile n has dim
//      16 g4 + 2 n in row g4 and 16 g4 + 2 n + 1 in row g4 + 8; the two keys of a register are
//      paired by a byte permute before the conversion.
//   Key row i of an 8-row group is key i, or i ^ 4 for odd i: with the 128-byte swizzle of the
//      boxes the eight lanes of a 16-byte load phase then touch all 32 banks, for K and for V.
#include "cache8.cuh"
#include "kernels.h"
#include "mma8.cuh"
#include "select.cuh"

namespace dash {

constexpr int kQ8Warps = 4;          // consumer warps per CTA
constexpr int kQ8Stages = 6;         // list entries (64 keys) in flight per CTA
constexpr int kQ8Keys = 32;          // keys per unit: a consumer's share of an entry
// An entry's two units fall to warps 0, 1 or 2, 3 by its parity, so an even ring gives every stage
// the same two consumers: each waits for a stage only after it has used the entry before, and
// the wait never meets a barrier that is still a phase behind.
static_assert(kQ8Warps == 4 && kQ8Stages % 2 == 0, "a stage keeps its consumers");
// An entry takes a CTA as long as about 3 CTAs' pieces (4 warps each) take a merge (split_ctas).  With 6
// entries a CTA always, lists of 1 to 6 blocks take 16.5 and 20.6 us a step against 14.4 and 16.5; with
// 2 always, two lists of 117 blocks 25.2 us against 21.1.
constexpr int kQ8Merge = 3;
constexpr int kQ8PartHead = 4;       // floats of a partial before its output: mA, sum, mB, -
constexpr float kWBits = 12.0f;      // weights reach 2^12: f16 then keeps terms down to 2^-36 of the largest

// What the consumers need to know of an entry, written by the producer beside its rows.
struct Q8Info {
    float lp[8];                     // log2 priors of the heads (-inf: block not selected, or no head)
    uint8_t scale[2][64];            // scale bytes of its keys and values
    int group, j, pad[2];
};
static_assert(sizeof(Q8Info) == 176, "slot of a stage: 16-byte rows");

template <int D>
struct Q8Layout {
    static constexpr uint32_t kPart = kBlock * D;               // K or V codes of one entry
    static constexpr uint32_t kStage = 2 * kPart;
    static constexpr uint32_t off_info = kQ8Stages * kStage;    // [stage] Q8Info
    static constexpr uint32_t kRow = kQ8PartHead + D;           // a partial
    static constexpr uint32_t bytes = off_info + kQ8Stages * (uint32_t)sizeof(Q8Info) + 1024;
    static_assert(2 * (bytes + 2048) <= 227 * 1024, "two CTAs share an SM");
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_e4m3(const float* f) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// a * b, at most the largest finite number (NaN stays NaN): the factors of a key and of a query may overflow
// together where their codes' product is zero, and the logit is zero then
__device__ __forceinline__ float mul_finite(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, 0f7F7FFFFF;" : "=f"(r) : "f"(a * b));
    return r;
}

template <int D>
__global__ void __launch_bounds__((kQ8Warps + 1) * 32, 2)
decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs,
                 const int* __restrict__ kv_len, const float* __restrict__ xs, const float* __restrict__ tau,
                 const int* __restrict__ list, const int* __restrict__ count, int* __restrict__ offs,
                 float* __restrict__ part, WsHeader* __restrict__ hdr, DecodeGeom g, int split, float e_pow, float sm2) {
    using L = Q8Layout<D>;
    using namespace sm100;
    constexpr int NT = D / 16;                       // 16-dim output tiles
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kQ8Stages], empty[kQ8Stages];
    __shared__ int abort_sh;
    __shared__ int share_sh[kQ8Warps + 4];
    const int cap = g.nbs + 1, cta = blockIdx.x;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const base_ptr = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        abort_sh = 0;
        for (int s = 0; s < kQ8Stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 2);
        }
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    pdl_wait();
    pdl_trigger();                                     // after the wait: the merge may read the lists at once
    // the barriers are visible after list_share's barriers
    const ListShare sh = list_share<(kQ8Warps + 1) * 32>(count, g.B * g.Hkv, cta, (int)gridDim.x, kQ8Merge, share_sh);
    if (tid == 0 && cta == 0) offs[g.B * g.Hkv] = sh.U;   // for the merge
    if (sh.lo >= sh.hi) return;                        // whole CTA: nothing listed for it
    volatile int* abort_flag = &abort_sh;

    if (warp == kQ8Warps) {
        // ------------------------------------------------------------ producer
        // One lane copies.  The warp walks the list four entries at a time, lane = (entry, head): it
        // turns their scores into the priors and brings the scale bytes (lane: 16 of the entry's
        // 128) that go with the rows, and loads the next four entries' meanwhile.  Copies take a
        // whole entry's keys or values: at 32 keys, with bulk copies for the scales, this loop
        // needed 1000 cycles for 8 KB, more than HBM does.
        const int hl = lane & 7, le = lane >> 3;
        long long cnt = 0;
        bool ok = true;
        for (int bg = sh.first, pos = sh.lo, o0 = sh.o_first, o1; ok && pos < sh.hi; ++bg, o0 = o1) {
            o1 = bg == sh.first ? sh.o_end : o0 + __ldcg(count + bg);
            if (o1 <= pos) continue;
            const int e_end = min(sh.hi, o1) - o0;
            if (pos == o0 && lane == 0) offs[bg] = o0;
            const int b = bg / g.Hkv, kvh = bg % g.Hkv, row0 = bg / split * g.Tmax;
            const int bt = (kv_len[b] - 1) / kBlock;
            const size_t qrow = (size_t)b * g.Hq + (size_t)kvh * g.G + (hl < g.G ? hl : 0);
            const float tu = __ldcg(tau + qrow);
            const float* xr = xs + qrow * cap;
            const int* lst = list + (size_t)bg * cap;
            auto entry = [&](int e) { return e < e_end ? __ldcg(lst + e) : 0; };
            int e0 = pos - o0;
            int j1 = entry(e0 + le), j2 = entry(e0 + 4 + le);    // these four entries' blocks, the next
            const uint8_t* sr = (hl < 4 ? ks : vs) + row0 + (hl & 3) * 16;
            auto scales = [&](int j) { return __ldg(reinterpret_cast<const uint4*>(sr + (size_t)j * kBlock)); };
            float x1 = __ldcg(xr + j1);
            uint4 s1 = scales(j1);
            for (; e0 < e_end && ok; e0 += 4) {
                const int j = j1;
                const float x = x1;
                const uint4 sc = s1;
                j1 = j2;
                x1 = __ldcg(xr + j1);
                s1 = scales(j1);
                j2 = entry(e0 + 8 + le);
                float lp = -INFINITY;
                if (hl < g.G) lp = j == bt ? 0.f : x > tu ? e_pow * __log2f(x - tu) : -INFINITY;
                const int n = min(4, e_end - e0);
                for (int i = 0; i < n; ++i, ++cnt) {
                    const int st = (int)(cnt % kQ8Stages), ji = __shfl_sync(0xffffffffu, j, i * 8);
                    if (cnt >= kQ8Stages) ok = mbar_wait(smem_u32(&empty[st]), (uint32_t)(((cnt / kQ8Stages) - 1) & 1), abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    Q8Info* info = reinterpret_cast<Q8Info*>(base_ptr + L::off_info) + st;
                    if (le == i) {
                        info->lp[hl] = lp;
                        *reinterpret_cast<uint4*>(&info->scale[hl >> 2][(hl & 3) * 16]) = sc;
                    }
                    if (lane == 0) { info->group = bg; info->j = ji; }
                    __syncwarp();
                    if (lane == 0) {
                        const int row = row0 + ji * kBlock;
                        const uint32_t dst = base + st * L::kStage, bar = smem_u32(&full[st]);
                        mbar_arrive_expect_tx(bar, L::kStage);
                        tma_load_2d(dst, &tm_k, 0, row, bar);
                        tma_load_2d(dst + L::kPart, &tm_v, 0, row, bar);
                    }
                }
            }
            pos = o0 + e_end;
        }
        if (lane == 0) {
            // the copies land before the CTA exits, also where a consumer gives up after the last was issued
            volatile int dummy = 0;
            for (int s = 0; s < kQ8Stages; ++s) {
                if (cnt <= s) continue;
                const long long last = cnt - 1 - ((cnt - 1 - s) % kQ8Stages);
                dummy = 0;
                mbar_wait(smem_u32(&full[s]), (uint32_t)((last / kQ8Stages) & 1), &dummy);
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumer warps
    // A warp takes every kQ8Warps-th unit of the CTA's range with a softmax state of its own, and
    // leaves it as a partial whenever the group changes: no warp waits for another.
    const int g4 = lane >> 2, t4 = lane & 3;
    const int kperm = (g4 & 1) ? g4 ^ 4 : g4;                           // key of MMA row g4
    const int units = 2 * (sh.hi - sh.lo);
    uint32_t qh[D / 32][2], ql[D / 32][2];                              // q' = hi + lo / 16 in e4m3
    float qf[2];                                                        // 2^e_q log2(e) / sqrt(d) of heads 2 t4, 2 t4 + 1
    float ma[2], mb[2], l_r[2], o[NT][4];
    int bg = -1, bt = 0, t = 0;
    // the partial of the group so far
    auto leave = [&]() {
        float* pw = part + (((size_t)cta + bg) * kQ8Warps + warp) * g.G * L::kRow;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int hl = 2 * t4 + hh;
            float l = l_r[hh];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (hl >= g.G) continue;
            float* pr = pw + (size_t)hl * L::kRow;
            if (g4 == 0) *reinterpret_cast<float4*>(pr) = make_float4(ma[hh], l, mb[hh], 0.f);
#pragma unroll
            for (int n = 0; n < NT; n += 2)
                *reinterpret_cast<float4*>(pr + kQ8PartHead + g4 * NT * 2 + 2 * n) = make_float4(o[n][hh], o[n][2 + hh], o[n + 1][hh], o[n + 1][2 + hh]);
        }
    };
    bool ok = true;
    for (int u = warp; u < units; u += kQ8Warps) {
        const int e = u >> 1, st = e % kQ8Stages;
        const bool got = ok && mbar_wait(smem_u32(&full[st]), (uint32_t)((e / kQ8Stages) & 1), abort_flag);
        if (!__all_sync(0xffffffffu, got)) { ok = false; continue; }
        const Q8Info* info = reinterpret_cast<const Q8Info*>(base_ptr + L::off_info) + st;
        const int j = info->j, group = info->group;
        const float2 lp = *reinterpret_cast<const float2*>(info->lp + 2 * t4);
        if (group != bg) {
            if (bg >= 0) leave();
            bg = group;
            const int b = bg / g.Hkv, kvh = bg % g.Hkv;
            t = kv_len[b] - 1;
            bt = t / kBlock;
            const size_t qrow0 = (size_t)b * g.Hq + (size_t)kvh * g.G;
            // B operand Q'^T: lane column g4 is the head; heads past G are zero
            uint4 w[D / 32];
            float amax = 0.f;
            int bad = 0;                                 // an element that is no number: the head's logits are NaN
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                w[c] = make_uint4(0u, 0u, 0u, 0u);
                if (g4 < g.G) w[c] = *(reinterpret_cast<const uint4*>(q + (qrow0 + g4) * D + (c >> 1) * 64 + t4 * 16) + (c & 1));
                float f[8];
                bf16x8_to_float(w[c], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool fin = fabsf(f[i]) < INFINITY;
                    amax = fmaxf(amax, fin ? fabsf(f[i]) : 0.f);
                    bad |= !fin;
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^-e_q in two factors (e_q may be as low as -140)
            const int eq = amax > 0.f ? ilogbf(amax) - 7 : 0;
            const int e1 = min(-eq, 127), e2 = -eq - e1;
            const float s1 = __uint_as_float((unsigned)(e1 + 127) << 23), s2 = __uint_as_float((unsigned)(e2 + 127) << 23);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float f[8];
                bf16x8_to_float(w[c], f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[k] = f[4 * i + k] * s1 * s2;
                    qh[c][i] = pack_e4m3(r);
                    float hv[4];
                    e4m3x4_to_float(qh[c][i], 1.0f, hv);
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[k] = (r[k] - hv[k]) * 16.0f;
                    ql[c][i] = pack_e4m3(r);
                }
            }
            // head h's factor sits on the lanes with g4 = h
            const unsigned bads = __ballot_sync(0xffffffffu, bad);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned lanes = 0xfu << ((2 * t4 + i) * 4);
                const int e = __shfl_sync(0xffffffffu, eq, (2 * t4 + i) * 4);
                qf[i] = bads & lanes ? __uint_as_float(0x7fc00000u) : scalbnf(sm2, e);
                ma[i] = mb[i] = -INFINITY;
                l_r[i] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[n][c] = 0.f;
        }
        {
            const int hk = u & 1;
            const bool diag = (j == bt);
            const uint32_t kst = base + st * L::kStage + hk * kQ8Keys * D, vst = kst + L::kPart;
            const uint8_t* ksc = info->scale[0] + hk * kQ8Keys;
            const uint8_t* vsc = info->scale[1] + hk * kQ8Keys;
            const int key0 = j * kBlock + hk * kQ8Keys;
            // S^T = K Q'^T
            // four accumulation chains: two key tiles x the two parts of q'
            float s[2][4], sl[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[mt][c] = sl[mt][c] = 0.f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                uint4 kr[2][2];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const int r0 = mt * 16 + kperm, r1 = r0 + 8;
                    // r1 & 7 == r0 & 7: both rows are swizzled alike
                    const int c0 = D == 128 ? (h * 4 + t4) ^ (r0 & 7) : t4 ^ ((r0 >> 1) & 3);
                    kr[mt][0] = lds128(kst + r0 * D + c0 * 16);
                    kr[mt][1] = lds128(kst + r1 * D + c0 * 16);
                }
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                    const int step = 2 * h + i2;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint32_t ka[4] = {i2 ? kr[mt][0].z : kr[mt][0].x, i2 ? kr[mt][1].z : kr[mt][1].x,
                                                i2 ? kr[mt][0].w : kr[mt][0].y, i2 ? kr[mt][1].w : kr[mt][1].y};
                        mma_e4m3(s[mt], ka, qh[step][0], qh[step][1]);
                        mma_e4m3(sl[mt], ka, ql[step][0], ql[step][1]);
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[mt][c] = fmaf(sl[mt][c], 0.0625f, s[mt][c]);
            // logits in log2 units; sb = logit + exponent of the key's value scale
            float sb[2][4], mxa[2] = {-INFINITY, -INFINITY}, mxb[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int key = mt * 16 + hh * 8 + kperm;
                    const float kf = scale_value(ksc[key]);
                    const unsigned sv = vsc[key];
                    const float ev = sv == kScaleNaN ? __uint_as_float(0x7fc00000u) : (float)((int)sv - 127);
                    const bool off = diag && key0 + key > t;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float p = c ? lp.y : lp.x;
                        const bool none = off || p == -INFINITY;
                        const float l2 = none ? -INFINITY : fmaf(s[mt][2 * hh + c], mul_finite(kf, qf[c]), p);
                        const float lb = none ? -INFINITY : l2 + ev;
                        s[mt][2 * hh + c] = l2;
                        sb[mt][2 * hh + c] = lb;
                        mxa[c] = fmaxf(mxa[c], l2);
                        mxb[c] = fmaxf(mxb[c], lb);
                    }
                }
            float mua[2], mub[2], sca[2], scb[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    mxa[c] = fmaxf(mxa[c], __shfl_xor_sync(0xffffffffu, mxa[c], off));
                    mxb[c] = fmaxf(mxb[c], __shfl_xor_sync(0xffffffffu, mxb[c], off));
                }
                const float na = fmaxf(ma[c], mxa[c]), nb = fmaxf(mb[c], mxb[c]);
                mua[c] = na == -INFINITY ? 0.f : na;
                mub[c] = nb == -INFINITY ? 0.f : nb;
                sca[c] = fast_exp2(ma[c] - mua[c]);
                scb[c] = fast_exp2(mb[c] - mub[c]);
                ma[c] = na;
                mb[c] = nb;
                mub[c] -= kWBits;
            }
            uint32_t pb[2][2];
            float ls[2] = {0.f, 0.f};
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) ls[c] += fast_exp2(s[mt][2 * hh + c] - mua[c]);
                    pb[mt][hh] = movmatrix_trans(pack_f16(fast_exp2(sb[mt][2 * hh] - mub[0]), fast_exp2(sb[mt][2 * hh + 1] - mub[1])));
                }
#pragma unroll
            for (int c = 0; c < 2; ++c) l_r[c] = l_r[c] * sca[c] + ls[c];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n][0] *= scb[0]; o[n][1] *= scb[1];
                o[n][2] *= scb[0]; o[n][3] *= scb[1];
            }
            // O^T += V^T W^T: two 16-key steps
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                constexpr int NW = D / 32;                       // words per lane and key
                uint32_t w[4][NW];
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const int k2 = 2 * t4 + (i4 & 1);
                    const int key = kk * 16 + (i4 >> 1) * 8 + ((i4 & 1) ? k2 ^ 4 : k2);
                    if constexpr (D == 128) {
                        const uint4 v = lds128(vst + key * 128 + ((g4 ^ (key & 7)) << 4));
                        w[i4][0] = v.x; w[i4][1] = v.y; w[i4][2] = v.z; w[i4][3] = v.w;
                    } else {
                        const uint2 v = lds64(vst + key * 64 + (((g4 >> 1) ^ ((key >> 1) & 3)) << 4) + (g4 & 1) * 8);
                        w[i4][0] = v.x; w[i4][1] = v.y;
                    }
                    // rows behind the sequence may hold anything, NaN codes too
                    if (diag && key0 + key > t) {
#pragma unroll
                        for (int c = 0; c < NW; ++c) w[i4][c] = 0u;
                    }
                }
#pragma unroll
                for (int c = 0; c < NW; ++c) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t sel = hf ? 0x7362u : 0x5140u;
                        const uint32_t x = __byte_perm(w[0][c], w[1][c], sel), y = __byte_perm(w[2][c], w[3][c], sel);
                        const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)x), e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                                               e4m3x2_to_f16x2((uint16_t)y), e4m3x2_to_f16x2((uint16_t)(y >> 16))};
                        mma_f16(o[2 * c + hf], a, pb[kk][0], pb[kk][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
        }
    }
    if (bg >= 0) leave();
    if (tid == 0 && *abort_flag) atomicOr(&hdr->status, kStWaitTimeout);
}

// One CTA of four warps per query head merges the partials of its group: every warp that had a
// unit of the group left one.  Where they lie follows from the lists' lengths, which are there before
// the attention ends; then the statistics and the first outputs are loaded together.
template <int D>
__global__ void __launch_bounds__(128)
decode_q8_combine_kernel(const int* __restrict__ count, const int* __restrict__ offs, const float* __restrict__ part,
                         __nv_bfloat16* __restrict__ out, DecodeGeom g, int nctas) {
    constexpr uint32_t kRow = Q8Layout<D>::kRow;
    constexpr int DPL = D / 32, KB = 8;                // KB: pieces whose loads are in flight together
    __shared__ float wt_sh[kDecodeMaxCtas * kQ8Warps], red[2][4], os[4][D];
    __shared__ int place_sh[8];
    const int bh = blockIdx.x, b = bh / g.Hq, h = bh % g.Hq, bg = b * g.Hkv + h / g.G, hl = h % g.G;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ListPlace at = list_place<128>(count, offs, g.B * g.Hkv, bg, place_sh);
    const ListSplit sp(at.U, g.B * g.Hkv, nctas, kQ8Merge);
    int c0 = 0, np = 0;
    if (at.n > 0) {
        c0 = sp.cta_of(at.o0);
        np = (sp.cta_of(at.o0 + at.n - 1) - c0 + 1) * kQ8Warps;
    }
    const float* p = part + ((size_t)(c0 + bg) * kQ8Warps * g.G + hl) * kRow;
    const size_t step = (size_t)g.G * kRow;
    // 1 where warp i % kQ8Warps of CTA c0 + i / kQ8Warps had one of the group's units
    for (int i = tid; i < np; i += 128) {
        const int c = c0 + i / kQ8Warps, w = i % kQ8Warps, lo = sp.lo(c), hi = sp.lo(c + 1);
        const int u0 = 2 * (max(lo, at.o0) - lo), u1 = 2 * (min(hi, at.o0 + at.n) - lo);
        wt_sh[i] = u0 + (w - u0 % kQ8Warps + kQ8Warps) % kQ8Warps < u1 ? 1.f : 0.f;
    }
    __syncthreads();
    pdl_wait();
    if (np == 0) return;                               // no keys: the select pass wrote zeros
    float v[KB][DPL];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int i = i0 + 4 * k;
#pragma unroll
            for (int d = 0; d < DPL; ++d) v[k][d] = 0.f;
            if (i < np && wt_sh[i] != 0.f) {
                const float* pi = p + i * step + kQ8PartHead + lane * DPL;
                if constexpr (DPL == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(pi));
                    v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(pi));
                    v[k][0] = x.x; v[k][1] = x.y;
                }
            }
        }
    };
    auto stats = [&](int i) {
        return i < np && wt_sh[i] != 0.f ? __ldcg(reinterpret_cast<const float4*>(p + i * step)) : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    };
    const float4 first = stats(tid);
    load(warp);
    float MA = first.x, MB = first.z;
    for (int i = tid + 128; i < np; i += 128) {
        const float4 s = stats(i);
        MA = fmaxf(MA, s.x);
        MB = fmaxf(MB, s.z);
    }
    MA = warp_max(MA);
    MB = warp_max(MB);
    if (lane == 0) { red[0][warp] = MA; red[1][warp] = MB; }
    __syncthreads();                                   // also: every warp has read its flags
    MA = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    MB = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
    const float ua = MA == -INFINITY ? 0.f : MA, ub = MB == -INFINITY ? 0.f : MB;
    float den = first.y * exp2f(first.x - ua);         // 0 where nothing was left (exp2 of -inf)
    for (int i = tid + 128; i < np; i += 128) {
        const float4 s = stats(i);
        den = fmaf(s.y, exp2f(s.x - ua), den);
        if (wt_sh[i] != 0.f) wt_sh[i] = exp2f(s.z - ub);
    }
    if (tid < np && wt_sh[tid] != 0.f) wt_sh[tid] = exp2f(first.z - ub);
    den = warp_sum(den);
    __syncthreads();
    if (lane == 0) red[0][warp] = den;
    float acc[DPL];
#pragma unroll
    for (int d = 0; d < DPL; ++d) acc[d] = 0.f;
    for (int i0 = warp;;) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int i = i0 + 4 * k;
            const float wk = i < np ? wt_sh[i] : 0.f;
#pragma unroll
            for (int d = 0; d < DPL; ++d) acc[d] = fmaf(v[k][d], wk, acc[d]);
        }
        i0 += 4 * KB;
        if (i0 >= np) break;
        load(i0);
    }
#pragma unroll
    for (int d = 0; d < DPL; ++d) os[warp][lane * DPL + d] = acc[d];
    __syncthreads();
    den = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
    // the partials' weights carry 2^kWBits and the values' maximum mB instead of mA
    const float f = den != 0.f ? exp2f(ub - ua - kWBits) / den : 0.f;
    if (tid < D) out[(size_t)bh * D + tid] = __float2bfloat16(((os[0][tid] + os[1][tid]) + (os[2][tid] + os[3][tid])) * f);
}

template <int D>
static cudaError_t launch_attn(const void* q, const void* kc, const void* vc, const void* ks, const void* vs,
                               const int* kv_len, void* out, const DecodeQ8Geom& gq, char* ws, float alpha, int nctas,
                               cudaStream_t stream) {
    const DecodeGeom& g = gq.v;
    CUtensorMap tk, tv;
    const unsigned long long rows = (unsigned long long)gq.real.B * gq.real.Hkv * g.Tmax;
    if (!make_tmap_u8(&tk, kc, rows, D, kBlock) || !make_tmap_u8(&tv, vc, rows, D, kBlock)) return cudaErrorInvalidValue;
    const int sm = (int)Q8Layout<D>::bytes;
    cudaError_t e = cudaFuncSetAttribute(decode_q8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    if (e != cudaSuccess) return e;
    const PdlConfig c(nctas, (kQ8Warps + 1) * 32, sm, stream);
    e = cudaLaunchKernelEx(&c.cfg, decode_q8_kernel<D>, tk, tv, static_cast<const __nv_bfloat16*>(q),
                           static_cast<const uint8_t*>(ks), static_cast<const uint8_t*>(vs), kv_len,
                           reinterpret_cast<const float*>(ws + g.off_x), reinterpret_cast<const float*>(ws + g.off_tau),
                           reinterpret_cast<const int*>(ws + g.off_list), reinterpret_cast<const int*>(ws + g.off_count),
                           reinterpret_cast<int*>(ws + g.off_offs), reinterpret_cast<float*>(ws + g.off_part),
                           reinterpret_cast<WsHeader*>(ws), g, gq.split, 1.0f / (alpha - 1.0f),
                           1.4426950408889634f / sqrtf((float)D));
    if (e != cudaSuccess) return e;
    const PdlConfig cc(g.B * g.Hq, 128, 0, stream);
    e = cudaLaunchKernelEx(&cc.cfg, decode_q8_combine_kernel<D>, reinterpret_cast<const int*>(ws + g.off_count),
                           reinterpret_cast<const int*>(ws + g.off_offs), reinterpret_cast<const float*>(ws + g.off_part),
                           static_cast<__nv_bfloat16*>(out), g, nctas);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_decode_q8(const void* q, const void* kc, const void* vc, const void* ks, const void* vs,
                             const float* ksum, const int* kv_len, void* out, const DecodeQ8Geom& g, char* ws,
                             float alpha, float coarse_scale, cudaStream_t stream) {
    const int nctas = decode_tc_ctas();
    cudaError_t e = launch_decode_lists(q, ksum, kv_len, out, g.real, g.v, ws, alpha, coarse_scale, 0, stream, true);
    if (e != cudaSuccess) return e;
    return g.v.d == 128 ? launch_attn<128>(q, kc, vc, ks, vs, kv_len, out, g, ws, alpha, nctas, stream)
                        : launch_attn<64>(q, kc, vc, ks, vs, kv_len, out, g, ws, alpha, nctas, stream);
}

}  // namespace dash
