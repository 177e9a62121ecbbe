// decode_q8.cu -- split-KV attention of a decode step over the 8-bit KV cache.
//
// The arithmetic of decode_tc.cu on the values that the cache holds (code 2^(s - 127),
// cache8.cuh), with the same balanced split over the concatenated block lists, the same
// segments, partials and merge.  What differs:
//
// Codes go to the tensor cores as f16, in which every e4m3 number is exact, with fp32 sums.
// The power-of-two scales stay outside the products:
//   K: logit = (q' . code) 2^(s_k - 127) 2^(e_q) / sqrt(d), q' = q 2^-e_q as f16 with the head's
//      largest magnitude in [2^14, 2^15): q's 8 significant bits are exact over 31 binades below
//      it, and what lies deeper is off by at most 2^-40 of the largest.
//   V: the weight that multiplies a key's codes is w = 2^(l + s_v - 127 - mB), l the logit (log2)
//      and mB the running maximum of l + s_v - 127 over the keys so far, so that w lies in
//      (0, 2^kWBits] whatever the scales are and its rounding to f16 (11 bits) is relative to
//      the largest contribution.  The softmax's sum has its own maximum mA over l.
// The sum takes the unrounded weights: w's rounding is 2^-12, far below bf16 output's 2^-9.
//
// Fragments straight from the codes.  A consumer computes S^T = K Q^T and O^T += V^T W^T with
// m16n8k16 (32 keys are two M tiles, the group's <= 8 heads the N columns), and the order of
// dims inside a contraction, of output rows, and of the keys of a unit is free, so a lane takes
// 16 consecutive bytes per shared-memory load:
//   K: slots (2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9) of step i are dims 16 t4 + 4 i + 0 .. 3 of the
//      64-dim half;
//   V: lane row g4 owns dims 16 g4 .. 16 g4 + 15 (d = 64: 8 g4 .. + 7): M tile n has dim
//      16 g4 + 2 n in row g4 and 16 g4 + 2 n + 1 in row g4 + 8; the two keys of a register are
//      paired by a byte permute before the conversion.
//   Key row i of an 8-row group is key i, or i ^ 4 for odd i: with the 128-byte swizzle of the
//      boxes the eight lanes of a 16-byte load phase then touch all 32 banks, for K and for V.
#include "cache8.cuh"
#include "kernels.h"
#include "mma_sync.cuh"
#include "select.cuh"
#include "sm100.cuh"

namespace dash {

constexpr int kQ8Warps = 4;          // consumer warps per CTA
constexpr int kQ8Stages = 8;         // units in flight per CTA (two per consumer warp)
constexpr int kQ8MaxG = 8;           // query heads per virtual group (one n8 tile)
constexpr int kQ8Keys = 32;          // keys per unit
constexpr int kQ8Tab = 64;           // list entries staged per table fill
constexpr int kQ8Per = 4;            // list entries per CTA at least
constexpr int kQ8PartHead = 4;       // floats of a partial before its output
constexpr float kWBits = 12.0f;      // weights reach 2^12: f16 then keeps terms down to 2^-36 of the largest

template <int D>
struct Q8Layout {
    static constexpr uint32_t kPart = kQ8Keys * D;              // K or V codes of one unit
    static constexpr uint32_t kStage = 2 * kPart;
    static constexpr uint32_t kTx = kStage + 2 * kQ8Keys;       // with the scale bytes
    static constexpr uint32_t off_scale = kQ8Stages * kStage;   // [stage][K 32, V 32]
    static constexpr uint32_t off_merge = off_scale + kQ8Stages * 2 * kQ8Keys;
    static constexpr uint32_t kRow = kQ8PartHead + D;           // mA, sum, mB, -, output
    static constexpr uint32_t merge_floats = kQ8Warps * kQ8MaxG * kRow > kDecodeMaxCtas * kQ8MaxG
                                                 ? kQ8Warps * kQ8MaxG * kRow : kDecodeMaxCtas * kQ8MaxG;
    static constexpr uint32_t off_tab = off_merge + merge_floats * 4;
    static constexpr uint32_t tab_bytes = kQ8Tab * kQ8MaxG * 4 + kQ8Tab * 4;
    static constexpr uint32_t bytes = off_tab + tab_bytes + 1024;
    static_assert(2 * (bytes + 2048) <= 227 * 1024, "two CTAs share an SM");
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
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
__device__ __forceinline__ unsigned lds8(uint32_t a) {
    unsigned v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

template <int D>
__global__ void __launch_bounds__((kQ8Warps + 1) * 32, 2)
decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs,
                 const int* __restrict__ kv_len, const float* __restrict__ xs, const float* __restrict__ tau,
                 const int* __restrict__ list, const int* __restrict__ count,
                 float* __restrict__ part, int* __restrict__ done, __nv_bfloat16* __restrict__ out,
                 WsHeader* __restrict__ hdr, DecodeGeom g, int split, float e_pow, float sm2) {
    using L = Q8Layout<D>;
    using namespace sm100;
    constexpr int T = kQ8Warps * 32;                 // consumer threads
    constexpr int NT = D / 16;                       // 16-dim output tiles
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kQ8Stages], empty[kQ8Stages];
    __shared__ int abort_sh, ticket_sh;
    __shared__ float wa_sh[kQ8Warps][kQ8MaxG], inv_sh[kQ8MaxG];
    __shared__ int share_sh[kQ8Warps + 3];
    const int cap = g.nbs + 1, cta = blockIdx.x;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const base_ptr = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        abort_sh = 0;
        for (int s = 0; s < kQ8Stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    pdl_wait();
    // the barriers are visible after list_share's barriers
    const ListShare sh = list_share<(kQ8Warps + 1) * 32>(count, g.B * g.Hkv, cta, (int)gridDim.x, kQ8Per, share_sh);
    if (sh.lo >= sh.hi) return;                        // whole CTA: nothing listed for it
    const long long U = sh.U;
    const int nC = sh.nC, r_hi = sh.hi;
    volatile int* abort_flag = &abort_sh;

    if (warp == kQ8Warps) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            long long cnt = 0;
            bool ok = true;
            for (int bg = sh.first, pos = sh.lo, o0 = sh.o_first, o1; ok && pos < r_hi; ++bg, o0 = o1) {
                o1 = o0 + __ldcg(count + bg);
                if (o1 <= pos) continue;
                const int seg_hi = min(r_hi, o1);
                for (int e = pos - o0; e < seg_hi - o0 && ok; ++e) {
                    const int j = list[(size_t)bg * cap + e];
                    for (int hk = 0; hk < 2; ++hk, ++cnt) {
                        const int st = (int)(cnt % kQ8Stages);
                        if (cnt >= kQ8Stages &&
                            !mbar_wait(smem_u32(&empty[st]), (uint32_t)(((cnt / kQ8Stages) - 1) & 1), abort_flag)) { ok = false; break; }
                        const int row = bg / split * g.Tmax + j * kBlock + hk * kQ8Keys;
                        const uint32_t dst = base + st * L::kStage, sdst = base + L::off_scale + st * 2 * kQ8Keys;
                        const uint32_t bar = smem_u32(&full[st]);
                        mbar_arrive_expect_tx(bar, L::kTx);
                        tma_load_2d(dst, &tm_k, 0, row, bar);
                        tma_load_2d(dst + L::kPart, &tm_v, 0, row, bar);
                        bulk_load_1d(sdst, ks + row, kQ8Keys, bar);
                        bulk_load_1d(sdst + kQ8Keys, vs + row, kQ8Keys, bar);
                    }
                }
                pos = seg_hi;
            }
            if (!ok) {
                // let the copies already issued land before the CTA exits
                volatile int dummy = 0;
                for (int s = 0; s < kQ8Stages; ++s) {
                    if (cnt <= s) continue;
                    const long long last = cnt - 1 - ((cnt - 1 - s) % kQ8Stages);
                    dummy = 0;
                    mbar_wait(smem_u32(&full[s]), (uint32_t)((last / kQ8Stages) & 1), &dummy);
                }
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumer warps
    const int g4 = lane >> 2, t4 = lane & 3;
    const int kperm = (g4 & 1) ? g4 ^ 4 : g4;                           // key of MMA row g4
    float* merge = reinterpret_cast<float*>(base_ptr + L::off_merge);   // [warp][head][kRow]
    float* lptab = reinterpret_cast<float*>(base_ptr + L::off_tab);     // [entry][8] log2 priors
    int* jtab = reinterpret_cast<int*>(base_ptr + L::off_tab + kQ8Tab * kQ8MaxG * 4);
    auto cons_sync = [&]() { asm volatile("bar.sync 1, %0;" :: "n"(T) : "memory"); };
    long long cnt = 0;
    bool ok = true;
    for (int bg = sh.first, pos = sh.lo, o0 = sh.o_first, o1; pos < r_hi; ++bg, o0 = o1) {
        o1 = o0 + __ldcg(count + bg);
        if (o1 <= pos) continue;
        const int seg_hi = min(r_hi, o1);
        const int e_lo = pos - o0, e_hi = seg_hi - o0;
        pos = seg_hi;
        const int b = bg / g.Hkv, kvh = bg % g.Hkv;
        const int t = kv_len[b] - 1, bt = t / kBlock;
        const size_t qrow0 = (size_t)b * g.Hq + (size_t)kvh * g.G;
        // B operand Q'^T: lane column g4 is the head; heads past G are zero
        uint32_t qb[D / 16][2];
        float qf[2];                                                    // 2^e_q log2(e) / sqrt(d) of heads 2 t4, 2 t4 + 1
        {
            uint4 w[D / 32];
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                w[c] = make_uint4(0u, 0u, 0u, 0u);
                if (g4 < g.G) w[c] = *(reinterpret_cast<const uint4*>(q + (qrow0 + g4) * D + (c >> 1) * 64 + t4 * 16) + (c & 1));
                float f[8];
                bf16x8_to_float(w[c], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]) < INFINITY ? fabsf(f[i]) : 0.f);
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^-e_q in two factors (e_q may be as low as -147): q' is exact whatever q's size
            const int eq = amax > 0.f ? ilogbf(amax) - 14 : 0;
            const int e1 = min(-eq, 127), e2 = -eq - e1;
            const float s1 = __uint_as_float((unsigned)(e1 + 127) << 23), s2 = __uint_as_float((unsigned)(e2 + 127) << 23);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float f[8];
                bf16x8_to_float(w[c], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = f[i] * s1 * s2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    qb[2 * c + i][0] = pack_f16(f[4 * i], f[4 * i + 1]);
                    qb[2 * c + i][1] = pack_f16(f[4 * i + 2], f[4 * i + 3]);
                }
            }
            // head h's factor sits on the lanes with g4 = h
#pragma unroll
            for (int i = 0; i < 2; ++i) qf[i] = scalbnf(sm2, __shfl_sync(0xffffffffu, eq, (2 * t4 + i) * 4));
        }
        // state of heads 2 t4 and 2 t4 + 1
        float ma[2] = {-INFINITY, -INFINITY}, mb[2] = {-INFINITY, -INFINITY}, l_r[2] = {0.f, 0.f};
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[n][c] = 0.f;

        for (int i0 = e_lo; i0 < e_hi; i0 += kQ8Tab) {
            const int nsub = min(kQ8Tab, e_hi - i0);
            cons_sync();                               // the previous table is no longer read
            for (int idx = tid; idx < nsub * kQ8MaxG; idx += T) {
                const int i = idx / kQ8MaxG, hl = idx % kQ8MaxG;
                const int j = list[(size_t)bg * cap + i0 + i];
                float v2 = -INFINITY;
                if (hl < g.G) {
                    if (j == bt) v2 = 0.f;
                    else {
                        const float x = xs[(qrow0 + hl) * cap + j], tu = tau[qrow0 + hl];
                        if (x > tu) v2 = e_pow * __log2f(x - tu);
                    }
                }
                lptab[idx] = v2;
                if (hl == 0) jtab[i] = j;
            }
            cons_sync();
            for (int i = 0; i < nsub; ++i) {
                // unit cnt (half hk of entry i) belongs to warp cnt % kQ8Warps
                for (int hk = 0; hk < 2; ++hk, ++cnt) {
                    if ((int)(cnt % kQ8Warps) != warp) continue;
                    const int j = jtab[i];
                    const bool diag = (j == bt);
                    const float2 lp = *reinterpret_cast<const float2*>(lptab + i * kQ8MaxG + 2 * t4);
                    const int st = (int)(cnt % kQ8Stages);
                    const bool got = ok && mbar_wait(smem_u32(&full[st]), (uint32_t)((cnt / kQ8Stages) & 1), abort_flag);
                    if (!__all_sync(0xffffffffu, got)) { ok = false; continue; }
                    const uint32_t kst = base + st * L::kStage, vst = kst + L::kPart;
                    const uint32_t sst = base + L::off_scale + st * 2 * kQ8Keys;
                    const int key0 = j * kBlock + hk * kQ8Keys;
                    // S^T = K Q'^T
                    float s[2][4];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[mt][c] = 0.f;
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) {
                            uint4 a0, a1;
                            const int r0 = mt * 16 + kperm, r1 = r0 + 8;
                            if constexpr (D == 128) {
                                const int c0 = (h * 4 + t4) ^ (r0 & 7);          // r1 & 7 == r0 & 7
                                a0 = lds128(kst + r0 * 128 + c0 * 16);
                                a1 = lds128(kst + r1 * 128 + c0 * 16);
                            } else {
                                const int c0 = t4 ^ ((r0 >> 1) & 3);
                                a0 = lds128(kst + r0 * 64 + c0 * 16);
                                a1 = lds128(kst + r1 * 64 + c0 * 16);
                            }
                            const uint32_t w0[4] = {a0.x, a0.y, a0.z, a0.w}, w1[4] = {a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                            for (int i4 = 0; i4 < 4; ++i4) {
                                const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)w0[i4]), e4m3x2_to_f16x2((uint16_t)w1[i4]),
                                                       e4m3x2_to_f16x2((uint16_t)(w0[i4] >> 16)),
                                                       e4m3x2_to_f16x2((uint16_t)(w1[i4] >> 16))};
                                mma_f16(s[mt], a, qb[h * 4 + i4][0], qb[h * 4 + i4][1]);
                            }
                        }
                    }
                    // logits in log2 units; sb = logit + exponent of the key's value scale
                    float sb[2][4], mxa[2] = {-INFINITY, -INFINITY}, mxb[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int key = mt * 16 + hh * 8 + kperm;
                            const float kf = scale_value(lds8(sst + key));
                            const unsigned sv = lds8(sst + kQ8Keys + key);
                            const float ev = sv == kScaleNaN ? __uint_as_float(0x7fc00000u) : (float)((int)sv - 127);
                            const bool off = diag && key0 + key > t;
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float p = c ? lp.y : lp.x;
                                const bool none = off || p == -INFINITY;
                                const float l2 = none ? -INFINITY : fmaf(s[mt][2 * hh + c], kf * qf[c], p);
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
                        sca[c] = exp2f(ma[c] - mua[c]);
                        scb[c] = exp2f(mb[c] - mub[c]);
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
                            for (int c = 0; c < 2; ++c) ls[c] += exp2f(s[mt][2 * hh + c] - mua[c]);
                            pb[mt][hh] = movmatrix_trans(pack_f16(exp2f(sb[mt][2 * hh] - mub[0]), exp2f(sb[mt][2 * hh + 1] - mub[1])));
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
        }
        // ---- merge the warps' states
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float l = l_r[hh];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int hl = 2 * t4 + hh;
            if (hl >= g.G) continue;
            float* mrow = merge + ((size_t)warp * kQ8MaxG + hl) * L::kRow;
            if (g4 == 0) { mrow[0] = ma[hh]; mrow[1] = l; mrow[2] = mb[hh]; }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mrow[kQ8PartHead + g4 * NT * 2 + 2 * n] = o[n][hh];
                mrow[kQ8PartHead + g4 * NT * 2 + 2 * n + 1] = o[n][2 + hh];
            }
        }
        cons_sync();
        const int c0 = dt_cta_of(o0, U, nC), c1 = dt_cta_of(o1 - 1, U, nC);
        const bool direct = (c0 == c1);
        const size_t slot = (size_t)cta + bg;
        if (tid < g.G) {
            float MA = -INFINITY, MB = -INFINITY;
#pragma unroll
            for (int w = 0; w < kQ8Warps; ++w) {
                const float* mrow = merge + ((size_t)w * kQ8MaxG + tid) * L::kRow;
                MA = fmaxf(MA, mrow[0]);
                MB = fmaxf(MB, mrow[2]);
            }
            const float ua = MA == -INFINITY ? 0.f : MA, ub = MB == -INFINITY ? 0.f : MB;
            float den = 0.f;
#pragma unroll
            for (int w = 0; w < kQ8Warps; ++w) {
                const float* mrow = merge + ((size_t)w * kQ8MaxG + tid) * L::kRow;
                den = fmaf(mrow[1], exp2f(mrow[0] - ua), den);
                wa_sh[w][tid] = exp2f(mrow[2] - ub);
            }
            // output = (sum of o 2^(mb - MB)) 2^(MB - MA - kWBits) / den
            inv_sh[tid] = den != 0.f ? exp2f(ub - ua - kWBits) / den : 0.f;
            if (!direct) {
                float* pr = part + (slot * g.G + tid) * L::kRow;
                *reinterpret_cast<float4*>(pr) = make_float4(MA, den, MB, 0.f);
            }
        }
        cons_sync();
        for (int idx = tid; idx < g.G * D; idx += T) {
            const int hl = idx / D, dim = idx % D;
            float acc = 0.f;
#pragma unroll
            for (int w = 0; w < kQ8Warps; ++w) acc = fmaf(merge[((size_t)w * kQ8MaxG + hl) * L::kRow + kQ8PartHead + dim], wa_sh[w][hl], acc);
            if (direct) out[(qrow0 + hl) * D + dim] = __float2bfloat16(acc * inv_sh[hl]);
            else part[(slot * g.G + hl) * L::kRow + kQ8PartHead + dim] = acc;
        }
        if (!direct) {
            // the CTA that writes the group's last piece merges all of them
            __threadfence();
            cons_sync();
            const int npieces = c1 - c0 + 1;
            if (tid == 0) ticket_sh = atomicAdd(&done[bg], 1);
            cons_sync();
            if (ticket_sh == npieces - 1) {
                __threadfence();
                // weights of the pieces, lanes over pieces; then the outputs, four dims per thread
                // and many pieces' loads in flight (a piece at a time this merge took 20 us of the
                // 16K step's 31)
                const float* p0 = part + ((size_t)c0 + bg) * g.G * L::kRow;
                const size_t pstep = (size_t)g.G * L::kRow;
                for (int hl = warp; hl < g.G; hl += kQ8Warps) {
                    float MA = -INFINITY, MB = -INFINITY, den = 0.f;
                    for (int pc = lane; pc < npieces; pc += 32) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(p0 + pc * pstep + hl * L::kRow));
                        MA = fmaxf(MA, v.x);
                        MB = fmaxf(MB, v.z);
                    }
                    MA = warp_max(MA);
                    MB = warp_max(MB);
                    const float ua = MA == -INFINITY ? 0.f : MA, ub = MB == -INFINITY ? 0.f : MB;
                    for (int pc = lane; pc < npieces; pc += 32) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(p0 + pc * pstep + hl * L::kRow));
                        den = fmaf(v.y, exp2f(v.x - ua), den);
                        merge[pc * g.G + hl] = exp2f(v.z - ub);
                    }
                    den = warp_sum(den);
                    if (lane == 0) inv_sh[hl] = den != 0.f ? exp2f(ub - ua - kWBits) / den : 0.f;
                }
                cons_sync();
                constexpr int NO = kQ8MaxG * D / 4 / T;
                float4 acc[NO];
#pragma unroll
                for (int k = 0; k < NO; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int pc = 0; pc < npieces; ++pc) {
#pragma unroll
                    for (int k = 0; k < NO; ++k) {
                        const int idx = tid + k * T, hl = idx / (D / 4), c = idx % (D / 4) * 4;
                        if (hl < g.G) {
                            const float4 v = __ldcg(reinterpret_cast<const float4*>(p0 + pc * pstep + hl * L::kRow + kQ8PartHead + c));
                            const float wt = merge[pc * g.G + hl];
                            acc[k].x = fmaf(v.x, wt, acc[k].x);
                            acc[k].y = fmaf(v.y, wt, acc[k].y);
                            acc[k].z = fmaf(v.z, wt, acc[k].z);
                            acc[k].w = fmaf(v.w, wt, acc[k].w);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < NO; ++k) {
                    const int idx = tid + k * T, hl = idx / (D / 4), c = idx % (D / 4) * 4;
                    if (hl < g.G) {
                        const float f = inv_sh[hl];
                        *reinterpret_cast<uint2*>(out + (qrow0 + hl) * D + c) = make_uint2(pack_bf16(acc[k].x * f, acc[k].y * f), pack_bf16(acc[k].z * f, acc[k].w * f));
                    }
                }
            }
        }
        cons_sync();                                  // the merge buffer is reused
    }
    if (tid == 0 && *abort_flag) atomicOr(&hdr->status, kStWaitTimeout);
}

template <int D>
static cudaError_t launch_attn(const void* q, const void* kc, const void* vc, const void* ks, const void* vs,
                               const int* kv_len, void* out, const DecodeQ8Geom& gq, char* ws, float alpha, int nctas,
                               cudaStream_t stream) {
    const DecodeGeom& g = gq.v;
    CUtensorMap tk, tv;
    const unsigned long long rows = (unsigned long long)gq.real.B * gq.real.Hkv * g.Tmax;
    if (!make_tmap_u8(&tk, kc, rows, D, kQ8Keys) || !make_tmap_u8(&tv, vc, rows, D, kQ8Keys)) return cudaErrorInvalidValue;
    const int sm = (int)Q8Layout<D>::bytes;
    cudaError_t e = cudaFuncSetAttribute(decode_q8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    if (e != cudaSuccess) return e;
    const PdlConfig c(nctas, (kQ8Warps + 1) * 32, sm, stream);
    e = cudaLaunchKernelEx(&c.cfg, decode_q8_kernel<D>, tk, tv, static_cast<const __nv_bfloat16*>(q),
                           static_cast<const uint8_t*>(ks), static_cast<const uint8_t*>(vs), kv_len,
                           reinterpret_cast<const float*>(ws + g.off_x), reinterpret_cast<const float*>(ws + g.off_tau),
                           reinterpret_cast<const int*>(ws + g.off_list), reinterpret_cast<const int*>(ws + g.off_count),
                           reinterpret_cast<float*>(ws + g.off_part), reinterpret_cast<int*>(ws + g.off_done),
                           static_cast<__nv_bfloat16*>(out), reinterpret_cast<WsHeader*>(ws), g, gq.split,
                           1.0f / (alpha - 1.0f), 1.4426950408889634f / sqrtf((float)D));
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
