// decode.cu -- one decode step of DashAttention with a split-KV (flash-decoding) layout.
//
// Same arithmetic as a prefill row t = kv_len - 1 ("DashAttention: Making Sparse Attention
// Fully Differentiable with Adaptive Block Selection", section "Core Mechanism"): coarse
// scores over the cached block summaries of blocks j < bt = t / 64, alpha-entmax weights,
// then softmax over the selected blocks' tokens plus the own block (causal, prior 1) with
// log p as the prior.  Kernels, all launched with shapes known on the host:
//   1. decode_scores : x[b, h, j] for every head of a KV group, each block summary read once
//                      for all G heads (a warp streams 16 summaries of one group);
//   2. decode_select : per (b, kv head): one warp per head solves tau with the row in shared
//                      memory, the union of the heads' selected blocks becomes the
//                      group's list (own block last), and the last CTA writes the work plan
//                      of the balanced attention pass;
//   3. attention     : decode_attn_tc_kernel (decode_tc.cu) for G <= 8, which also merges
//                      the split groups; otherwise decode_attn below, split-KV over chunks of
//                      16 listed blocks with a two-stage cp.async pipeline, each listed block
//                      read once for every head of the group, partial (max, sum, output) per
//                      chunk and head, and
//   4. decode_combine: merging those partials of each (b, h) into bf16.
// The HBM traffic that matters is step 3: (union blocks + 1) * 64 * d * 2 bytes * 2 per
// (b, kv head).
#include <cstdlib>
#include <cstring>

#include "common.cuh"
#include "entmax.cuh"
#include "kernels.h"
#include "select.cuh"

namespace dash {

// ------------------------------------------------------------------ scores
//
// x[b, h, j] = cx * q[b, h] . kbar[b, g, j] for the G heads of every group and every past
// block j < bt.  A warp takes RW consecutive block summaries of one group and issues all
// their loads at once (lane l holds dims [l D/32, (l + 1) D/32) of each row: one coalesced
// row per instruction); the group's query rows sit in registers (heads padded to GP, a
// power of two <= 8).  Per task of R = 32/GP rows (at most 8) a lane has R * GP partial sums,
// and a butterfly reduce-scatter over the 32 lanes leaves every (row, head) sum complete on
// its own lane with 31 shuffles in all.  Each summary is read from HBM once for all heads.

// Butterfly reduce-scatter of C values per lane over lane offsets O, O/2, ..., 1: at each
// level the lane with bit O set keeps the upper half of its values and receives the
// partner's copy of it; once one value is left, the remaining levels sum it.
template <int C, int O>
__device__ __forceinline__ void reduce_scatter(float* v, int lane) {
    if constexpr (O >= 1) {
        if constexpr (C >= 2) {
            const bool up = (lane & O) != 0;
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                const float send = up ? v[i] : v[i + C / 2];
                const float keep = up ? v[i + C / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, O);
            }
            reduce_scatter<C / 2, O / 2>(v, lane);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
            reduce_scatter<1, O / 2>(v, lane);
        }
    }
}

template <int D, int GP>
struct ScoreShape {
    static constexpr int DPL = D / 32;                 // dims per lane
    static constexpr int R = GP >= 4 ? 32 / GP : 8;    // rows per reduce-scatter
    static constexpr int V = R * GP;                   // partial sums per lane (<= 32)
    static constexpr int RW = 2 * R;                   // rows per warp, loads issued together
    static constexpr int LOGV = V >= 32 ? 5 : V >= 16 ? 4 : V >= 8 ? 3 : V >= 4 ? 2 : V >= 2 ? 1 : 0;
};

// The first block of a step's first kernel clears the workspace header (hdr null: the caller did).
__device__ __forceinline__ void clear_header(WsHeader* hdr, bool first) {
    if (hdr && first && threadIdx.x < sizeof(WsHeader) / 16) reinterpret_cast<uint4*>(hdr)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
}

// CTAs of two warps: at 97 registers a thread more of them fit an SM than of eight, and a short step's
// tasks reach more SMs (8 x 96K: 13.2 us against 13.6; an 8-bit step at 16K 21.8 against 22.8).
constexpr int kScoreThreads = 64;

template <int D, int GP>
__global__ void __launch_bounds__(kScoreThreads)
decode_scores_kernel(const __nv_bfloat16* __restrict__ q, const float* __restrict__ ksum,
                     const int* __restrict__ kv_len, float* __restrict__ xs, DecodeGeom g, float cx,
                     WsHeader* __restrict__ hdr) {
    using S = ScoreShape<D, GP>;
    clear_header(hdr, blockIdx.x == 0);
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long wtask = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int tpg = (g.nbs + S::RW - 1) / S::RW;
    const int bg = (int)(wtask / tpg);
    if (bg >= g.B * g.Hkv) return;
    const int j0 = (int)(wtask % tpg) * S::RW;
    const int b = bg / g.Hkv, kvh = bg % g.Hkv;
    const int L = kv_len[b];
    if (L < 1 || L > g.Tmax) return;
    const int bt = (L - 1) / kBlock;
    if (j0 >= bt) return;
    const size_t qrow0 = (size_t)b * g.Hq + (size_t)kvh * g.G;
    // rows past bt load row bt - 1 again (in bounds; their sums are not written)
    const float* src = ksum + (size_t)bg * g.nbs * D + lane * S::DPL;
    float kv[S::RW][S::DPL];
#pragma unroll
    for (int r = 0; r < S::RW; ++r) {
        const size_t jr = (size_t)min(j0 + r, bt - 1);
        if constexpr (S::DPL == 4) {
            const float4 t = __ldg(reinterpret_cast<const float4*>(src + jr * D));
            kv[r][0] = t.x; kv[r][1] = t.y; kv[r][2] = t.z; kv[r][3] = t.w;
        } else {
            const float2 t = __ldg(reinterpret_cast<const float2*>(src + jr * D));
            kv[r][0] = t.x; kv[r][1] = t.y;
        }
    }
    // query rows of the group (heads past G repeat head 0; their sums are not written)
    float qv[GP][S::DPL];
#pragma unroll
    for (int h = 0; h < GP; ++h) {
        const __nv_bfloat16* qh = q + (qrow0 + (h < g.G ? h : 0)) * D + lane * S::DPL;
        if constexpr (S::DPL == 4) {
            const uint2 t = __ldg(reinterpret_cast<const uint2*>(qh));
            const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&t.x));
            const float2 c = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&t.y));
            qv[h][0] = a.x; qv[h][1] = a.y; qv[h][2] = c.x; qv[h][3] = c.y;
        } else {
            const uint32_t t = __ldg(reinterpret_cast<const unsigned int*>(qh));
            const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&t));
            qv[h][0] = a.x; qv[h][1] = a.y;
        }
    }
    const size_t cap = (size_t)g.nbs + 1;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float v[S::V];
#pragma unroll
        for (int r = 0; r < S::R; ++r)
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                float acc = 0.f;
#pragma unroll
                for (int d = 0; d < S::DPL; ++d) acc = fmaf(kv[half * S::R + r][d], qv[h][d], acc);
                v[r * GP + h] = acc;
            }
        reduce_scatter<S::V, 16>(v, lane);
        // value index held by this lane (see reduce_scatter): lane * V/32 + k when V >= 32,
        // else lane >> (5 - log2 V), replicated on 32/V lanes
        if constexpr (S::V >= 32) {
#pragma unroll
            for (int k = 0; k < S::V / 32; ++k) {
                const int idx = lane * (S::V / 32) + k, r = idx / GP, h = idx % GP;
                const int j = j0 + half * S::R + r;
                if (h < g.G && j < bt) xs[(qrow0 + h) * cap + j] = v[k] * cx;
            }
        } else {
            const int idx = lane >> (5 - S::LOGV), r = idx / GP, h = idx % GP;
            const int j = j0 + half * S::R + r;
            if ((lane & ((32 >> S::LOGV) - 1)) == 0 && h < g.G && j < bt) xs[(qrow0 + h) * cap + j] = v[0] * cx;
        }
    }
}

// Groups of more than 8 heads: four threads per block summary, each with a quarter of its d
// values; every head's partial dot product is reduced over the four threads with two
// shuffles.
template <int D>
__global__ void __launch_bounds__(256)
decode_scores_wide_kernel(const __nv_bfloat16* __restrict__ q, const float* __restrict__ ksum,
                          const int* __restrict__ kv_len, float* __restrict__ xs, DecodeGeom g, float cx,
                          WsHeader* __restrict__ hdr) {
    clear_header(hdr, blockIdx.x == 0 && blockIdx.y == 0);
    pdl_trigger();
    constexpr int QD = D / 4;                 // dims per thread
    constexpr int QV = QD / 4;                // float4 per thread
    constexpr int QS = D + 16;                // padded row stride of a query head (floats)
    __shared__ __align__(16) float qs[32 * QS];
    const int bg = blockIdx.x, b = bg / g.Hkv, kvh = bg % g.Hkv;
    const int L = kv_len[b];
    if (L < 1 || L > g.Tmax) return;
    const int bt = (L - 1) / kBlock;
    const int j0 = blockIdx.y * 64;
    if (j0 >= bt) return;
    const int part = threadIdx.x & 3, j = j0 + (threadIdx.x >> 2);
    float4 kv[QV];
#pragma unroll
    for (int i = 0; i < QV; ++i) kv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < bt) {
        const float4* kb = reinterpret_cast<const float4*>(ksum + ((size_t)bg * g.nbs + j) * D + part * QD);
#pragma unroll
        for (int i = 0; i < QV; ++i) kv[i] = __ldg(kb + i);
    }
    for (int i = threadIdx.x; i < g.G * D; i += blockDim.x) {
        const int h = i / D, c = i % D;
        qs[h * QS + (c / QD) * (QD + 4) + c % QD] = __bfloat162float(q[(size_t)(b * g.Hq + kvh * g.G) * D + i]);
    }
    __syncthreads();
    const int cap = g.nbs + 1;
    for (int h0 = 0; h0 < g.G; h0 += 4) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) {
            if (h0 + hh >= g.G) break;
            const float4* qv = reinterpret_cast<const float4*>(qs + (h0 + hh) * QS + part * (QD + 4));
#pragma unroll
            for (int i = 0; i < QV; ++i) {
                const float4 a = qv[i];
                acc[hh] = fmaf(a.x, kv[i].x, acc[hh]);
                acc[hh] = fmaf(a.y, kv[i].y, acc[hh]);
                acc[hh] = fmaf(a.z, kv[i].z, acc[hh]);
                acc[hh] = fmaf(a.w, kv[i].w, acc[hh]);
            }
        }
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) {
            acc[hh] += __shfl_xor_sync(0xffffffffu, acc[hh], 1);
            acc[hh] += __shfl_xor_sync(0xffffffffu, acc[hh], 2);
        }
        const int h = h0 + part;
        const float mine = part == 0 ? acc[0] : part == 1 ? acc[1] : part == 2 ? acc[2] : acc[3];
        if (h < g.G && j < bt) xs[(size_t)(b * g.Hq + kvh * g.G + h) * cap + j] = mine * cx;
    }
}

template <int D, int GP>
void launch_scores_gp(const __nv_bfloat16* q, const float* ksum, const int* kv_len, float* xs,
                      const DecodeGeom& g, float cx, WsHeader* hdr, cudaStream_t stream) {
    using S = ScoreShape<D, GP>;
    const long long warps = (long long)g.B * g.Hkv * ((g.nbs + S::RW - 1) / S::RW);
    const unsigned grid = (unsigned)((warps + kScoreThreads / 32 - 1) / (kScoreThreads / 32));
    if (grid > 0) decode_scores_kernel<D, GP><<<grid, kScoreThreads, 0, stream>>>(q, ksum, kv_len, xs, g, cx, hdr);
}

template <int D>
void launch_scores(const __nv_bfloat16* q, const float* ksum, const int* kv_len, float* xs,
                   const DecodeGeom& g, float cx, WsHeader* hdr, cudaStream_t stream) {
    if (g.G == 1) launch_scores_gp<D, 1>(q, ksum, kv_len, xs, g, cx, hdr, stream);
    else if (g.G == 2) launch_scores_gp<D, 2>(q, ksum, kv_len, xs, g, cx, hdr, stream);
    else if (g.G <= 4) launch_scores_gp<D, 4>(q, ksum, kv_len, xs, g, cx, hdr, stream);
    else if (g.G <= 8) launch_scores_gp<D, 8>(q, ksum, kv_len, xs, g, cx, hdr, stream);
    else {
        dim3 gs(g.B * g.Hkv, (g.nbs + 63) / 64 > 0 ? (g.nbs + 63) / 64 : 1);
        decode_scores_wide_kernel<D><<<gs, 256, 0, stream>>>(q, ksum, kv_len, xs, g, cx, hdr);
    }
}

// ------------------------------------------------------------------ select

// One CTA of 8 warps per (b, kv head).  Warp w solves the thresholds of heads w, w + 8, ...
// with the row in shared memory, scap values of it at most (one warp per head: no cross-warp
// reduction in a pass).  The heads' selected blocks are OR-ed into a bitmap, which becomes the
// group's list, the own block last.
constexpr int kSelThreads = 256;

__global__ void __launch_bounds__(kSelThreads)
decode_select_kernel(const __nv_bfloat16* __restrict__ q, const int* __restrict__ kv_len, const float* __restrict__ xs,
                     float* __restrict__ tau, int* __restrict__ list, int* __restrict__ count,
                     int* __restrict__ done, int* __restrict__ offs, int* __restrict__ plan,
                     __nv_bfloat16* __restrict__ out, WsHeader* __restrict__ hdr, DecodeGeom g,
                     float alpha, int nctas, int hist_init, bool warm, int scap) {
    constexpr int kWords = kMaxT / kBlock / 32;
    __shared__ HistBins hist[kSelThreads / 32];
    __shared__ unsigned bitmap[kWords];
    __shared__ int list_sh[33 * (kSelThreads / 32)];
    extern __shared__ __align__(16) float rows_sm[];   // rows in 16-byte chunks
    const int bg = blockIdx.x, b = bg / g.Hkv, kvh = bg % g.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = kSelThreads / 32;
    const int cap = g.nbs + 1;
    const int L = kv_len[b];
    const size_t qrow0 = (size_t)b * g.Hq + (size_t)kvh * g.G;
    pdl_trigger();
    pdl_wait();
    if (tid == 0) done[bg] = 0;
    if (L < 1 || L > g.Tmax) {
        // no keys: the group's heads get a zero output and no work
        if (tid == 0) count[bg] = 0;
        for (int i = tid; i < g.G * g.d; i += kSelThreads) out[qrow0 * g.d + i] = __float2bfloat16(0.f);
        if (nctas > 0) decode_plan_tail(count, offs, plan, hdr, g.B * g.Hkv, nctas);
        return;
    }
    const int bt = (L - 1) / kBlock;
    const int nw = (bt + 31) / 32;
    for (int i = tid; i < nw; i += kSelThreads) bitmap[i] = 0u;
    __syncthreads();
    int no_conv = 0;
    for (int hl = warp; hl < g.G; hl += nwarp) {
        const size_t row = qrow0 + hl;
        WarpRow xr;
        xr.load(xs + row * cap, rows_sm + (size_t)warp * scap, scap, lane, bt);
        float t = __int_as_float(0x7fc00000);
        const float y = xr.lane_max(), m = warp_max(y);
        // warm, the 8-bit step: a head whose query is no number has nothing to solve and selects nothing (dash_decode
        // reports such a step as not converged)
        if (bt > 0 && !(warm && !(fabsf(m) < INFINITY) && row_not_finite(q + row * g.d, g.d)))
            t = row_tau(xr, m, alpha, &no_conv, hist_init ? &hist[warp] : nullptr, g.maxit, warm ? lane_start(y - m, alpha) : -1.0f);
        if (lane == 0) tau[row] = t;
        const int nsel = xr.words(t, [&](int k, unsigned w) { atomicOr(&bitmap[k], w); });
        if (lane == 0) {
            atomicAdd(&hdr->selected_pairs, (unsigned long long)nsel);
            atomicAdd(&hdr->scored_pairs, (unsigned long long)bt);
        }
    }
    if (no_conv) atomicOr(&hdr->status, kStNoConverge);
    __syncthreads();
    int* dst = list + (size_t)bg * cap;
    const int total = bits_to_list([&](int i) { return bitmap[i]; }, nw, dst, list_sh, nwarp);
    if (tid == 0) {
        dst[total] = bt;                  // own block, always last
        count[bg] = total + 1;
        atomicAdd(&hdr->union_blocks, (unsigned long long)total);
        if (bt > 0) atomicAdd(&hdr->tiles, 1ull);
    }
    if (nctas > 0) decode_plan_tail(count, offs, plan, hdr, g.B * g.Hkv, nctas);
}

template <int D>
__device__ __forceinline__ int swz_d(int row, int c) { return row * D + ((c ^ (row & 7)) << 3); }

template <int D>
__global__ void __launch_bounds__(128)
decode_attn_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kc,
                   const __nv_bfloat16* __restrict__ vc, const int* __restrict__ kv_len,
                   const float* __restrict__ xs, const float* __restrict__ tau,
                   const int* __restrict__ list, const int* __restrict__ count,
                   float* __restrict__ part, DecodeGeom g, float e_pow, float sm2) {
    constexpr int CH = D / 8;
    extern __shared__ uint4 smem_u4[];
    __nv_bfloat16* Ks = reinterpret_cast<__nv_bfloat16*>(smem_u4);   // [2][64][D]
    __nv_bfloat16* Vs = Ks + 2 * kBlock * D;                          // [2][64][D]
    float* qs = reinterpret_cast<float*>(Vs + 2 * kBlock * D);       // [G][D]
    float* os = qs + g.G * D;                                         // [G][D]
    float* ls = os + g.G * D;                                         // [G][64] logits, then p
    float* m_s = ls + g.G * kBlock;                                   // [G]
    float* l_s = m_s + 32;                                            // [G]
    float* sc_s = l_s + 32;                                           // [G]
    float* lp_s = sc_s + 32;                                          // [G]

    const int bg = blockIdx.x, b = bg / g.Hkv, kvh = bg % g.Hkv;
    const int n = count[bg];
    const int e0 = blockIdx.y * g.chunk;
    if (e0 >= n) return;
    const int e1 = min(n, e0 + g.chunk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = kv_len[b];
    const int t = L - 1, bt = t / kBlock;
    const int cap = g.nbs + 1;
    const int* lst = list + (size_t)bg * cap;
    const size_t row0 = (size_t)bg * g.Tmax;

    auto load_kv = [&](int e, int stage) {
        const int j = lst[e];
        for (int idx = tid; idx < kBlock * CH; idx += blockDim.x) {
            const int r = idx / CH, c = idx % CH;
            const int tok = j * kBlock + r;
            const bool ok = tok < L;
            const size_t off = (row0 + (ok ? tok : 0)) * D + c * 8;
            cp_async16(Ks + stage * kBlock * D + swz_d<D>(r, c), kc + off, ok ? 16 : 0);
            cp_async16(Vs + stage * kBlock * D + swz_d<D>(r, c), vc + off, ok ? 16 : 0);
        }
    };
    load_kv(e0, 0);
    cp_async_commit();
    for (int i = tid; i < g.G * D; i += blockDim.x) {
        qs[i] = __bfloat162float(q[(size_t)(b * g.Hq + kvh * g.G) * D + i]);
        os[i] = 0.f;
    }
    if (tid < g.G) { m_s[tid] = -INFINITY; l_s[tid] = 0.f; }

    for (int e = e0; e < e1; ++e) {
        const int stage = (e - e0) & 1;
        const int j = lst[e];
        const bool diag = (j == bt);
        if (e + 1 < e1) load_kv(e + 1, stage ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
        if (tid < g.G) {
            const size_t row = (size_t)(b * g.Hq + kvh * g.G + tid);
            float lp = 0.f;
            if (!diag) {
                const float x = xs[row * cap + j], ta = tau[row];
                lp = x > ta ? e_pow * __log2f(x - ta) : -INFINITY;
            }
            lp_s[tid] = lp;
        }
        __syncthreads();
        const __nv_bfloat16* Kst = Ks + stage * kBlock * D;
        const __nv_bfloat16* Vst = Vs + stage * kBlock * D;
        // logits: thread -> (key, head parity)
        {
            const int key = tid & 63;
            const bool masked = diag && (j * kBlock + key > t);
            for (int hl = tid >> 6; hl < g.G; hl += 2) {
                float acc = 0.f;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint4 u = *reinterpret_cast<const uint4*>(Kst + swz_d<D>(key, c));
                    float f[8];
                    bf16x8_to_float(u, f);
                    const float* qq = qs + hl * D + c * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc = fmaf(qq[i], f[i], acc);
                }
                const float lp = lp_s[hl];
                ls[hl * kBlock + key] = (masked || lp == -INFINITY) ? -INFINITY : fmaf(acc, sm2, lp);
            }
        }
        __syncthreads();
        // online softmax per head (one warp per head)
        for (int hl = warp; hl < g.G; hl += 4) {
            float a0 = ls[hl * kBlock + lane], a1 = ls[hl * kBlock + lane + 32];
            const float mx = warp_max(fmaxf(a0, a1));
            const float m_old = m_s[hl];
            const float m_new = fmaxf(m_old, mx);
            const float m_use = m_new == -INFINITY ? 0.f : m_new;
            a0 = exp2f(a0 - m_use);
            a1 = exp2f(a1 - m_use);
            const float sum = warp_sum(a0 + a1);
            ls[hl * kBlock + lane] = a0;
            ls[hl * kBlock + lane + 32] = a1;
            __syncwarp();
            if (lane == 0) {
                const float sc = exp2f(m_old - m_use);
                sc_s[hl] = sc;
                l_s[hl] = l_s[hl] * sc + sum;
                m_s[hl] = m_new;
            }
        }
        __syncthreads();
        // O = O * scale + P V : thread -> (head, pair of dims)
        for (int pidx = tid; pidx < g.G * (D / 2); pidx += blockDim.x) {
            const int hl = pidx / (D / 2), dp = pidx % (D / 2);
            const int dim = dp * 2, c = dim >> 3, off = dim & 7;
            float ax = 0.f, ay = 0.f;
            const float* p = ls + hl * kBlock;
#pragma unroll 8
            for (int key = 0; key < kBlock; ++key) {
                const __nv_bfloat162 vv = *reinterpret_cast<const __nv_bfloat162*>(
                    Vst + key * D + (((c ^ (key & 7)) << 3) + off));
                const float2 vf = __bfloat1622float2(vv);
                ax = fmaf(p[key], vf.x, ax);
                ay = fmaf(p[key], vf.y, ay);
            }
            const float sc = sc_s[hl];
            os[hl * D + dim] = fmaf(os[hl * D + dim], sc, ax);
            os[hl * D + dim + 1] = fmaf(os[hl * D + dim + 1], sc, ay);
        }
        __syncthreads();
    }
    // partial (m, l, o) for every head of the group
    const size_t pbase = ((size_t)bg * g.maxchunks + blockIdx.y) * g.G;
    for (int i = tid; i < g.G * (D + 2); i += blockDim.x) {
        const int hl = i / (D + 2), c = i % (D + 2);
        const float val = c == 0 ? m_s[hl] : (c == 1 ? l_s[hl] : os[hl * D + c - 2]);
        part[(pbase + hl) * (D + 2) + c] = val;
    }
}

template <int D>
__global__ void __launch_bounds__(128)
decode_combine_kernel(const int* __restrict__ count, const float* __restrict__ part,
                      __nv_bfloat16* __restrict__ out, DecodeGeom g) {
    const int bh = blockIdx.x, b = bh / g.Hq, h = bh % g.Hq;
    const int kvh = h / g.G, hl = h % g.G, bg = b * g.Hkv + kvh;
    const int n = count[bg];
    const int nch = (n + g.chunk - 1) / g.chunk;
    float M = -INFINITY;
    for (int c = 0; c < nch; ++c)
        M = fmaxf(M, part[(((size_t)bg * g.maxchunks + c) * g.G + hl) * (D + 2)]);
    const float Mu = M == -INFINITY ? 0.f : M;
    for (int dim = threadIdx.x; dim < D; dim += blockDim.x) {
        float num = 0.f, den = 0.f;
        for (int c = 0; c < nch; ++c) {
            const float* p = part + (((size_t)bg * g.maxchunks + c) * g.G + hl) * (D + 2);
            const float w = exp2f(p[0] - Mu);
            den = fmaf(p[1], w, den);
            num = fmaf(p[2 + dim], w, num);
        }
        out[(size_t)bh * D + dim] = __float2bfloat16(nch > 0 && den > 0.f ? num / den : 0.f);
    }
}

cudaError_t launch_decode_lists(const void* q, const float* ksum, const int* kv_len, void* out, const DecodeGeom& g,
                                const DecodeGeom& gl, char* ws, float alpha, float coarse_scale, int nctas,
                                cudaStream_t stream, bool pdl) {
    const float cx = (alpha - 1.0f) * coarse_scale / sqrtf((float)g.d);
    float* xs = reinterpret_cast<float*>(ws + gl.off_x);
    const auto* qb = static_cast<const __nv_bfloat16*>(q);
    WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
    if (g.d == 128) launch_scores<128>(qb, ksum, kv_len, xs, g, cx, pdl ? hdr : nullptr, stream);
    else launch_scores<64>(qb, ksum, kv_len, xs, g, cx, pdl ? hdr : nullptr, stream);
    // DASH_ENTMAX_INIT=histogram starts each threshold solve at the histogram edge; the
    // default, Newton from u = -1, is faster on the rows measured here (the binning pass
    // costs more than the passes it saves)
    const char* init = getenv("DASH_ENTMAX_INIT");
    const int hist_init = (init && strcmp(init, "histogram") == 0) ? 1 : 0;
    const int rows = gl.G < kSelThreads / 32 ? gl.G : kSelThreads / 32;            // rows that a CTA holds at a time
    const int fit = kSelBytes / (rows * (int)sizeof(float)) & ~31;
    const int scap = gl.nbs < fit ? gl.nbs : fit;
    const int sm = scap * rows * (int)sizeof(float);
    // the attribute is the function's, not the call's: another host thread's shorter cache must not lower it
    cudaError_t e = cudaFuncSetAttribute(decode_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelBytes);
    if (e != cudaSuccess) return e;
    PdlConfig c(gl.B * gl.Hkv, kSelThreads, sm, stream);
    if (!pdl) c.cfg.numAttrs = 0;
    e = cudaLaunchKernelEx(&c.cfg, decode_select_kernel, qb, kv_len, (const float*)xs, reinterpret_cast<float*>(ws + gl.off_tau),
                           reinterpret_cast<int*>(ws + gl.off_list), reinterpret_cast<int*>(ws + gl.off_count),
                           reinterpret_cast<int*>(ws + gl.off_done), reinterpret_cast<int*>(ws + gl.off_offs),
                           reinterpret_cast<int*>(ws + gl.off_plan), static_cast<__nv_bfloat16*>(out), hdr, gl, alpha, nctas,
                           hist_init, pdl, scap);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_decode(const void* q, const void* kc, const void* vc, const float* ksum,
                          const int* kv_len, void* out, const DecodeGeom& g, char* ws,
                          float alpha, float coarse_scale, cudaStream_t stream,
                          const cudaEvent_t* events, int agg, float* x_dump, float* p_dump) {
    auto mark = [&](int i) {
        return !events || cudaEventRecord(events[i], stream) == cudaSuccess;
    };
    const float e_pow = 1.0f / (alpha - 1.0f);
    const float sm2 = 1.4426950408889634f / sqrtf((float)g.d);
    float* xs = reinterpret_cast<float*>(ws + g.off_x);
    float* tau = reinterpret_cast<float*>(ws + g.off_tau);
    int* list = reinterpret_cast<int*>(ws + g.off_list);
    int* count = reinterpret_cast<int*>(ws + g.off_count);
    float* part = reinterpret_cast<float*>(ws + g.off_part);
    const auto* qb = static_cast<const __nv_bfloat16*>(q);
    const auto* kb = static_cast<const __nv_bfloat16*>(kc);
    const auto* vb = static_cast<const __nv_bfloat16*>(vc);
    auto* ob = static_cast<__nv_bfloat16*>(out);
    const int BH = g.B * g.Hkv;
    const bool fused = decode_tc_supported(g);
    const int nctas = fused ? decode_tc_ctas() : 0;
    cudaError_t e = cudaSuccess;
    if (!mark(0)) return cudaErrorUnknown;
    e = launch_decode_lists(q, ksum, kv_len, out, g, g, ws, alpha, coarse_scale, nctas, stream);
    if (e != cudaSuccess) return e;
    if (!mark(1)) return cudaErrorUnknown;
    if (fused) {
        e = launch_decode_attn_tc(q, kc, vc, kv_len, out, g, ws, e_pow, sm2, nctas, stream, agg, x_dump, p_dump);
        if (e != cudaSuccess) return e;
        if (!mark(2) || !mark(3)) return cudaErrorUnknown;   // no separate merge pass
        return cudaGetLastError();
    }
    // the CUDA-core path has per-head priors only and no parity dump
    if (agg || x_dump) return cudaErrorNotSupported;
    auto attn_bytes = [&](int G) {
        return (size_t)4 * kBlock * g.d * sizeof(__nv_bfloat16) + (size_t)(2 * G * g.d + G * kBlock + 4 * 32) * sizeof(float);
    };
    const size_t sm_attn = attn_bytes(g.G);
    // the attribute is the function's: always the size for the most heads, so no other thread's call lowers it
    const int sm_max = (int)attn_bytes(32);
    e = g.d == 128
        ? cudaFuncSetAttribute(decode_attn_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm_max)
        : cudaFuncSetAttribute(decode_attn_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm_max);
    if (e != cudaSuccess) return e;
    dim3 ga(BH, g.maxchunks);
    if (g.d == 128)
        decode_attn_kernel<128><<<ga, 128, sm_attn, stream>>>(qb, kb, vb, kv_len, xs, tau, list, count, part, g, e_pow, sm2);
    else
        decode_attn_kernel<64><<<ga, 128, sm_attn, stream>>>(qb, kb, vb, kv_len, xs, tau, list, count, part, g, e_pow, sm2);
    if (!mark(2)) return cudaErrorUnknown;
    if (g.d == 128) decode_combine_kernel<128><<<g.B * g.Hq, 128, 0, stream>>>(count, part, ob, g);
    else decode_combine_kernel<64><<<g.B * g.Hq, 128, 0, stream>>>(count, part, ob, g);
    if (!mark(3)) return cudaErrorUnknown;
    return cudaGetLastError();
}

}  // namespace dash
