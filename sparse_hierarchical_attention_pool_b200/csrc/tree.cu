// tree.cu -- one decode step for a tree of drafted tokens per sequence.
//
// Node i of sequence b (parent[b, i] < i, -1: a root) stands at position t = L + depth(i),
// L = kv_len[b], and attends as a decode step at t would if the tokens of its path (its
// ancestors and itself) followed the L cached ones ("DashAttention: Making Sparse Attention
// Fully Differentiable with Adaptive Block Selection", section "Core Mechanism").  With
// F = L / 64 full blocks and r = L % 64 tokens in the open block F:
//   - blocks j < F are past blocks, scored against their cached summaries;
//   - while r + depth < 64 the open block is the node's own block: its r cached tokens and the
//     whole path, prior 1;
//   - from r + depth >= 64 on, the path's first 64 - r tokens complete the open block, which is
//     then a past block whose summary is the mean of its r cached and 64 - r path keys
//     (different for every path), and the rest of the path is the own block.  With at most 64
//     nodes no path reaches a second end of a block.
// Kernels:
//   1. tree_scores : x[row, j] = cx q . kbar_j for the full blocks on the tensor cores, and in one
//                    CTA per KV group the ancestor masks, depths and the open block's scores;
//   2. tree_select : thresholds (one warp per row) and the union of every tile's selected blocks;
//   3. tree_attn, tree_combine (tree_tc.cu): every row over its selected blocks, the open block and
//                    its path.
#include "cache8.cuh"
#include "kernels.h"
#include "mma_sync.cuh"
#include "select.cuh"
#include "tree.cuh"

namespace dash {

// ------------------------------------------------------------------ scores
//
// 64 summaries per CTA, 16 per warp as the M rows of mma.sync m16n8k16, 8 query rows as the N
// columns.  kbar is split into bf16 hi + lo parts (16 significant bits; the products with bf16
// q are exact and summed in fp32), as in the prefill's coarse stage.  The k index of a step is
// a free permutation of the dims, so each lane loads 8 consecutive dims of its row at once:
// slots (2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9) of steps 2 c and 2 c + 1 are dims
// 32 c + 8 t4 + 0 .. 7.
// 96K, 8 sequences of 8 KV heads and 64 rows (50 MB of summaries, 25 MB of scores): 23 us, the latency of
// load, conversion and products in 2.6 waves of CTAs; 5 or 6 CTAs an SM instead of 4 spill (+4, +19 us).
constexpr int kScoreRows = 64;       // query rows per CTA

template <int D>
__device__ __forceinline__ void tree_score_chunk(const __nv_bfloat16* q, const float* ksum, float* xs, const TreeGeom& g,
                                                 int bg, int F, int j0, float cx) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int jw = j0 + warp * 16;
    if (jw >= F) return;
    uint32_t hi[D / 16][4], lo[D / 16][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int j = min(jw + g4 + 8 * half, F - 1);              // past F: row F - 1 again, not written
        const float4* src = reinterpret_cast<const float4*>(ksum + ((size_t)bg * g.nbs + j) * D) + t4 * 2;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float4 v = __ldg(src + c * 8 + s);
                const uint32_t h0 = pack_bf16(v.x, v.y), h1 = pack_bf16(v.z, v.w);
                const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h0));
                const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h1));
                hi[2 * c + s][half] = h0;
                hi[2 * c + s][2 + half] = h1;
                lo[2 * c + s][half] = pack_bf16(v.x - f0.x, v.y - f0.y);
                lo[2 * c + s][2 + half] = pack_bf16(v.z - f1.x, v.w - f1.y);
            }
        }
    }
    const size_t row0 = (size_t)bg * g.R;                           // rows of a KV group are contiguous in q
    const int r_lo = (int)blockIdx.z * kScoreRows, r_hi = min(g.R, r_lo + kScoreRows);
    auto load_q = [&](uint4 (&v)[D / 32], int r0) {
        const uint4* qr = reinterpret_cast<const uint4*>(q + (row0 + min(r0 + g4, g.R - 1)) * D) + t4;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) v[c] = __ldg(qr + c * 4);
    };
    uint4 v[D / 32], nv[D / 32];
    load_q(v, r_lo);
    for (int r0 = r_lo; r0 < r_hi; r0 += 8) {
        load_q(nv, r0 + 8);                                         // the next rows on their way
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            mma_bf16(acc, hi[2 * c], v[c].x, v[c].y);
            mma_bf16(acc, lo[2 * c], v[c].x, v[c].y);
            mma_bf16(acc, hi[2 * c + 1], v[c].z, v[c].w);
            mma_bf16(acc, lo[2 * c + 1], v[c].z, v[c].w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 2 * t4 + (i & 1), j = jw + g4 + 8 * (i >> 1);
            if (r < r_hi && j < F) xs[(row0 + r) * g.cap + j] = acc[i] * cx;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) v[c] = nv[c];
    }
}

// Row y = 0 of the grid prepares a KV group: ancestor sets, depths, the tiles' empty bitmaps and,
// where some path completes the open block, the mean of the open block's keys on every path.
template <int D, bool Q8>
__global__ void __launch_bounds__(128)
tree_scores_kernel(TreeArgs a, TreeWork w, TreeGeom g, float cx) {
    constexpr int TPR = D / 4, NR = 128 / TPR;                      // threads of 4 dims for a row, rows at once
    __shared__ int par_s[kMaxNodes];
    constexpr int KR = D + 8;                                       // a row of keys: 16 bytes on, so that 8 rows' chunks miss each other's banks
    __shared__ unsigned long long sum_s[kMaxNodes];
    __shared__ __align__(16) __nv_bfloat16 key_s[kMaxNodes][KR];
    __shared__ __align__(16) float tail_s[NR][D], tot_s[D];
    __shared__ unsigned in_s[kMaxNodes / 32];
    const int bg = blockIdx.x, b = bg / g.Hkv, tid = threadIdx.x;
    pdl_trigger();
    if (bg == 0 && blockIdx.y == 0 && blockIdx.z == 0 && tid < (int)sizeof(WsHeader) / 16)
        reinterpret_cast<uint4*>(w.hdr)[tid] = make_uint4(0u, 0u, 0u, 0u);
    if (blockIdx.y == 0 && tid < g.N) par_s[tid] = a.parent[(size_t)b * g.N + tid];
    int L, nodes;
    const bool live = tree_live(a.kv_len, a.n_nodes, g, b, &L, &nodes);
    const int F = live ? L / kBlock : 0;
    if (blockIdx.y > 0) {
        const int j0 = ((int)blockIdx.y - 1) * 64;
        if (j0 < F) tree_score_chunk<D>(static_cast<const __nv_bfloat16*>(a.q), a.ksum, w.xs, g, bg, F, j0, cx);
        return;
    }
    if (blockIdx.z > 0) return;
    // the group's tiles start with nothing selected
    for (int i = tid; i < g.tiles_bg * g.nbw; i += 128) w.bits[(size_t)bg * g.tiles_bg * g.nbw + i] = 0u;
    for (int i = tid; i < g.tiles_bg; i += 128) w.tick[bg * g.tiles_bg + i] = 0;
    // Some path may complete the open block (a path has at most `nodes` tokens): the draft's keys are on
    // their way while the paths are walked.
    const int r = live ? L % kBlock : 0;
    const bool may_cross = r + nodes > kBlock;
    if (may_cross) {
        const auto* kd = static_cast<const __nv_bfloat16*>(a.k_draft) + (size_t)bg * g.N * D;
        for (int i = tid; i < (nodes + 15) / 16 * 16 * (D / 8); i += 128) {
            const int row = i / (D / 8), ch = i % (D / 8) * 8;
            cp_async16(&key_s[row][ch], kd + (size_t)min(row, nodes - 1) * D + ch, row < nodes ? 16 : 0);   // zeros past the nodes
        }
    }
    // every node walks up its path (parents come before children, so the walk ends); a parent
    // outside [-1, i) makes the node and its descendants invalid
    __syncthreads();
    unsigned long long m = 0ull;
    int dp = -1;
    if (tid < nodes && live) {
        int i = tid;
        while (i >= 0) {
            const int p = par_s[i];
            if (p < -1 || p >= i) { m = 0ull; dp = -1; break; }
            m |= 1ull << i;
            ++dp;
            i = p;
        }
    }
    if (tid < g.N && bg % g.Hkv == 0) { w.anc[(size_t)b * g.N + tid] = m; w.depth[(size_t)b * g.N + tid] = dp; }
    if (!__syncthreads_or(may_cross && r + dp >= kBlock)) {
        cp_async_done();                                            // the copies land before the CTA's memory is another's
        return;
    }
    const int c = tid % TPR * 4, r0 = tid / TPR;
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr float kPart = 1.0f / kBlock;                          // exact: large keys must not add up to infinity
    const size_t row0 = (size_t)bg * g.Tmax + (L - r);
#pragma unroll 16
    for (int i = r0; i < r; i += NR) {
        float f[4];
        if constexpr (Q8) {
            e4m3x4_to_float(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.k_cache) + (row0 + i) * D + c),
                            scale_value(static_cast<const uint8_t*>(a.k_scale)[row0 + i]), f);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.k_cache) + (row0 + i) * D + c);
            const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
            const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
            f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = fmaf(f[k], kPart, t[k]);
    }
    // A path's mean: the cached keys of the open block and the path's tokens in it, those with
    // r + depth < 64 (the first 64 - r of a path, so they are bits of its ancestor set).  All of them
    // at once are one product of the 0 / 2^-6 ancestor matrix and the keys (exact products, fp32 sums): a
    // warp takes 16 nodes, in place of a walk of up to 64 dependent additions (4 us, now 1).
    const unsigned in_w = __ballot_sync(0xffffffffu, dp >= 0 && r + dp < kBlock);
    if (tid < kMaxNodes && (tid & 31) == 0) in_s[tid >> 5] = in_w;
    *reinterpret_cast<float4*>(&tail_s[r0][c]) = make_float4(t[0], t[1], t[2], t[3]);
    cp_async_done();
    __syncthreads();
    const unsigned long long in = in_s[0] | (unsigned long long)in_s[1] << 32;
    if (tid < kMaxNodes) sum_s[tid] = m & in;
    if (tid < D) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < NR; ++k) v += tail_s[k][tid];           // a fixed order
        tot_s[tid] = v;
    }
    __syncthreads();
    const int lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
    if (warp * 16 >= nodes) return;
    const int n0 = warp * 16 + g4, n1 = n0 + 8;
    const unsigned long long a0 = sum_s[n0], a1 = sum_s[n1];
    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[n][k] = 0.f;
    unsigned odd = 0u;                                              // a key that is no number
    for (int k0 = 0; k0 < nodes; k0 += 16) {
        // two bits as two bf16: 2^-6 or 0
        auto pair = [&](unsigned long long bits, int k) { return ((unsigned)(bits >> k) & 1u) * 0x3c80u | ((unsigned)(bits >> (k + 1)) & 1u) * 0x3c800000u; };
        const int k = k0 + 2 * t4;
        const uint32_t af[4] = {pair(a0, k), pair(a1, k), pair(a0, k + 8), pair(a1, k + 8)};
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            uint32_t bf[4];
            ldsm_x4_t(bf[0], bf[1], bf[2], bf[3], smem_u32(&key_s[k0 + (lane & 15)][n * 16 + (lane >> 4) * 8]));
#pragma unroll
            for (int q = 0; q < 4; ++q) odd |= __vcmpeq2(bf[q] & 0x7f807f80u, 0x7f807f80u);
            mma_bf16(acc[2 * n], af, bf[0], bf[1]);
            mma_bf16(acc[2 * n + 1], af, bf[2], bf[3]);
        }
    }
    float* dst = w.path + (size_t)bg * g.N * D;
    if (__any_sync(0xffffffffu, odd != 0u)) {
        // 0 times a key that is no number would reach nodes off its path: node by node
        for (int i = warp * 16; i < min(nodes, warp * 16 + 16); ++i)
            for (int e = lane; e < D; e += 32) {
                float v = tot_s[e];
                for (unsigned long long up = sum_s[i]; up; up &= up - 1) v = fmaf(__bfloat162float(key_s[__ffsll((long long)up) - 1][e]), kPart, v);
                dst[(size_t)i * D + e] = v;
            }
        return;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
        const float2 v = *reinterpret_cast<const float2*>(&tot_s[n * 8 + 2 * t4]);
        if (n0 < nodes) *reinterpret_cast<float2*>(dst + (size_t)n0 * D + n * 8 + 2 * t4) = make_float2(v.x + acc[n][0], v.y + acc[n][1]);
        if (n1 < nodes) *reinterpret_cast<float2*>(dst + (size_t)n1 * D + n * 8 + 2 * t4) = make_float2(v.x + acc[n][2], v.y + acc[n][3]);
    }
}

// ------------------------------------------------------------------ select
//
// One warp per row solves its threshold; every selected block sets its bit in the tile's bitmap
// (a ballot over the lanes is one word).  The CTA that finishes a tile turns the bitmap into
// the tile's list: selected full blocks ascending, the open block when it holds cached tokens
// (whether past or own), the tree itself last.  The latency of the passes over a row bounds it (no pipe above a quarter):
// 4,096 rows of 1,536 scores take 14 us and the lists 3.
constexpr int kTreeSelWarps = 8;

__global__ void __launch_bounds__(kTreeSelWarps * 32)
tree_select_kernel(TreeArgs a, TreeWork w, TreeGeom g, float alpha, float cx) {
    __shared__ int last_sh, list_sh[33 * kTreeSelWarps];
    extern __shared__ __align__(16) float rows_sm[];   // rows in 16-byte chunks
    const int scap = min(g.cap, kSelCap);
    constexpr int kCtasPerTile = kTreeRows / kTreeSelWarps;
    const int tile = blockIdx.x / kCtasPerTile, sub = blockIdx.x % kCtasPerTile;
    const int bg = tile / g.tiles_bg, b = bg / g.Hkv;
    const int r0 = (tile % g.tiles_bg) * kTreeRows, rows = min(kTreeRows, g.R - r0);
    if (sub * kTreeSelWarps >= rows) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int L, nodes;
    const bool live = tree_live(a.kv_len, a.n_nodes, g, b, &L, &nodes);
    const int F = live ? L / kBlock : 0, r = live ? L % kBlock : 0;
    pdl_trigger();
    pdl_wait();
    const int lrow = sub * kTreeSelWarps + warp;                     // row of the tile
    if (lrow < rows) {
        const size_t row = (size_t)bg * g.R + r0 + lrow;
        const int node = (r0 + lrow) % g.N;
        const int dp = w.depth[(size_t)b * g.N + node];
        if (node < (a.n_nodes ? min(a.n_nodes[b], g.N) : g.N) && (!live || dp < 0)) {
            // no valid length or parent: zero output
            for (int c = lane; c < g.d; c += 32) static_cast<__nv_bfloat16*>(a.out)[row * g.d + c] = __float2bfloat16(0.f);
        }
        float t = __int_as_float(0x7fc00000);
        if (live && dp >= 0) {
            const bool crossed = r + dp >= kBlock;
            int n = F + (crossed ? 1 : 0);
            float* xrow = w.xs + row * g.cap;
            if (crossed) {
                // the path completes the open block: its score from the mean of the block's 64 keys
                const auto* qr = static_cast<const __nv_bfloat16*>(a.q) + row * g.d;
                const float* pr = w.path + ((size_t)bg * g.N + node) * g.d;
                float s = 0.f;
                for (int c = lane; c < g.d; c += 32) s = fmaf(__bfloat162float(qr[c]), pr[c], s);
                s = warp_sum(s) * cx;
                // a path with a key that is no number has no such score: NaN, which makes the row NaN in the
                // attention, and no part of the threshold (it has no root then)
                if (!(fabsf(s) < INFINITY)) { s = __int_as_float(0x7fc00000); n = F; }
                if (lane == 0) xrow[F] = s;
                __syncwarp();
            }
            int no_conv = 0, nsel = 0;
            WarpRow xr;
            xr.load(xrow, rows_sm + (size_t)warp * scap, scap, lane, n);
            const float y = xr.lane_max(), m = warp_max(y);
            if (m > -INFINITY && !(m == INFINITY && row_not_finite(static_cast<const __nv_bfloat16*>(a.q) + row * g.d, g.d)))
                t = row_tau(xr, m, alpha, &no_conv, nullptr, g.maxit, lane_start(y - m, alpha));
            nsel = xr.words(t, [&](int k, unsigned sel) { atomicOr(&w.bits[(size_t)tile * g.nbw + k], sel); });
            if (lane == 0) {
                if (no_conv) atomicOr(&w.hdr->status, kStNoConverge);
                atomicAdd(&w.hdr->selected_pairs, (unsigned long long)nsel);
                atomicAdd(&w.hdr->scored_pairs, (unsigned long long)n);
            }
        }
        if (lane == 0) w.tau[row] = t;
    }
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        last_sh = atomicAdd(&w.tick[tile], 1) == (rows + kTreeSelWarps - 1) / kTreeSelWarps - 1;
    }
    __syncthreads();
    if (!last_sh) return;
    __threadfence();
    int* dst = w.list + (size_t)tile * g.lcap;
    int total = 0;
    if (live) {
        // the open block has its own entry
        auto word = [&](int i) {
            const unsigned m = __ldcg(w.bits + (size_t)tile * g.nbw + i);
            return i == F / 32 ? m & ((1u << (F & 31)) - 1u) : m;
        };
        total = bits_to_list(word, (F + 31) / 32, dst, list_sh, kTreeSelWarps);
        if (tid == 0) {
            atomicAdd(&w.hdr->union_blocks, (unsigned long long)total);
            if (total > 0) atomicAdd(&w.hdr->tiles, 1ull);
            if (r > 0) dst[total++] = kTreeOpen;
            dst[total++] = kTreeDraft;
        }
    }
    if (tid == 0) w.count[tile] = total;
}

// ------------------------------------------------------------------ host side

// one CTA per SM (its operand rings fill the shared memory)
static int tree_ctas() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n < 1 ? 1 : n < kDecodeMaxCtas ? n : kDecodeMaxCtas;
}

template <int D, bool Q8>
static cudaError_t launch_tree_t(const TreeArgs& a, const TreeGeom& g, char* ws, float alpha, float coarse_scale,
                                 cudaStream_t stream) {
    const float cx = (alpha - 1.0f) * coarse_scale / sqrtf((float)D);
    const float e_pow = 1.0f / (alpha - 1.0f), sm2 = 1.4426950408889634f / sqrtf((float)D);
    const TreeWork w = tree_work(g, ws);
    const dim3 gs((unsigned)(g.B * g.Hkv), (unsigned)((g.nbs + 63) / 64 + 1), (unsigned)((g.R + kScoreRows - 1) / kScoreRows));
    const int nctas = tree_ctas();
    tree_scores_kernel<D, Q8><<<gs, 128, 0, stream>>>(a, w, g, cx);
    const int sm = (g.cap < kSelCap ? g.cap : kSelCap) * kTreeSelWarps * (int)sizeof(float);
    // the attribute is the function's, not the call's: another host thread's shorter cache must not lower it
    cudaError_t e = cudaFuncSetAttribute(tree_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSelCap * kTreeSelWarps * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    const PdlConfig c((unsigned)g.tiles * (kTreeRows / kTreeSelWarps), kTreeSelWarps * 32, sm, stream);
    e = cudaLaunchKernelEx(&c.cfg, tree_select_kernel, a, w, g, alpha, cx);
    if (e != cudaSuccess) return e;
    return launch_tree_attn(a, w, g, e_pow, sm2, nctas, stream);
}

cudaError_t launch_tree(const TreeArgs& a, const TreeGeom& g, char* ws, float alpha, float coarse_scale, cudaStream_t stream) {
    if (g.d == 128) return a.k_scale ? launch_tree_t<128, true>(a, g, ws, alpha, coarse_scale, stream)
                                     : launch_tree_t<128, false>(a, g, ws, alpha, coarse_scale, stream);
    return a.k_scale ? launch_tree_t<64, true>(a, g, ws, alpha, coarse_scale, stream)
                     : launch_tree_t<64, false>(a, g, ws, alpha, coarse_scale, stream);
}

}  // namespace dash
