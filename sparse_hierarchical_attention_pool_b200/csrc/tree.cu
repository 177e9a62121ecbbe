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
//   2. tree_select : thresholds (one warp per row), the union of every tile's selected blocks,
//                    and the work plan;
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
    for (int r0 = 0; r0 < g.R; r0 += 8) {
        const int rq = min(r0 + g4, g.R - 1);
        const uint4* qr = reinterpret_cast<const uint4*>(q + (row0 + rq) * D) + t4;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 v = __ldg(qr + c * 4);
            mma_bf16(acc, hi[2 * c], v.x, v.y);
            mma_bf16(acc, lo[2 * c], v.x, v.y);
            mma_bf16(acc, hi[2 * c + 1], v.z, v.w);
            mma_bf16(acc, lo[2 * c + 1], v.z, v.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 2 * t4 + (i & 1), j = jw + g4 + 8 * (i >> 1);
            if (r < g.R && j < F) xs[(row0 + r) * g.cap + j] = acc[i] * cx;
        }
    }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(128)
tree_scores_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kd,
                   const int* __restrict__ parent, const int* __restrict__ n_nodes, const void* __restrict__ kc,
                   const uint8_t* __restrict__ ks, const float* __restrict__ ksum, const int* __restrict__ kv_len,
                   float* __restrict__ xs, unsigned long long* __restrict__ anc, int* __restrict__ depth,
                   unsigned* __restrict__ bits, int* __restrict__ tick, TreeGeom g, float cx) {
    __shared__ int par_s[kMaxNodes], dep_s[kMaxNodes];
    __shared__ float path[kMaxNodes][D];
    const int bg = blockIdx.x, b = bg / g.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int L, nodes;
    const bool live = tree_live(kv_len, n_nodes, g, b, &L, &nodes);
    const int F = live ? L / kBlock : 0;
    if (blockIdx.y > 0) {
        const int j0 = ((int)blockIdx.y - 1) * 64;
        if (j0 < F) tree_score_chunk<D>(q, ksum, xs, g, bg, F, j0, cx);
        return;
    }
    // the group's tiles start with nothing selected
    for (int i = tid; i < g.tiles_bg * g.nbw; i += 128) bits[(size_t)bg * g.tiles_bg * g.nbw + i] = 0u;
    for (int i = tid; i < g.tiles_bg; i += 128) tick[bg * g.tiles_bg + i] = 0;
    // ancestor sets and depths: every node walks up its path (parents come before children, so
    // the walk ends); a parent outside [-1, i) makes the node and its descendants invalid
    for (int i = tid; i < nodes; i += 128) par_s[i] = parent[(size_t)b * g.N + i];
    __syncthreads();
    if (tid < g.N) {
        unsigned long long a = 0ull;
        int dp = -1;
        if (live && tid < nodes) {
            int i = tid;
            while (i >= 0) {
                const int p = par_s[i];
                if (p < -1 || p >= i) { a = 0ull; dp = -1; break; }
                a |= 1ull << i;
                ++dp;
                i = p;
            }
        }
        dep_s[tid] = dp;
        if (bg % g.Hkv == 0) { anc[(size_t)b * g.N + tid] = a; depth[(size_t)b * g.N + tid] = dp; }
    }
    __syncthreads();
    if (!live) return;
    const int r = L % kBlock;
    int any = 0;
    for (int i = tid; i < nodes; i += 128) any |= r + dep_s[i] >= kBlock;
    any = __syncthreads_or(any);
    const size_t row0 = (size_t)bg * g.R;
    if (any) {
        // path[i] = the sum of the open block's keys on node i's path (all its tokens with
        // r + depth < 64), every dim a recurrence over the nodes
        for (int c = tid; c < D; c += 128) {
            float tail = 0.f;
            for (int t = L - r; t < L; ++t) {
                const size_t o = ((size_t)bg * g.Tmax + t);
                if constexpr (Q8) {
                    float f[4];
                    e4m3x4_to_float(static_cast<const uint8_t*>(kc)[o * D + c], scale_value(ks[o]), f);
                    tail += f[0];
                } else {
                    tail += __bfloat162float(static_cast<const __nv_bfloat16*>(kc)[o * D + c]);
                }
            }
            for (int i = 0; i < nodes; ++i) {
                const int p = par_s[i];
                if (dep_s[i] < 0) continue;
                float v = p >= 0 ? path[p][c] : tail;
                if (r + dep_s[i] < kBlock) v += __bfloat162float(kd[((size_t)bg * g.N + i) * D + c]);
                path[i][c] = v;
            }
        }
        __syncthreads();
    }
    for (int row = warp; row < g.R; row += 4) {
        const int node = row % g.N;
        const bool crossed = node < nodes && dep_s[node] >= 0 && r + dep_s[node] >= kBlock;
        float x = -INFINITY;
        if (crossed) {
            float s = 0.f;
            for (int c = lane; c < D; c += 32) s = fmaf(__bfloat162float(q[(row0 + row) * D + c]), path[node][c], s);
            x = warp_sum(s) * (cx / kBlock);
        }
        if (lane == 0) xs[(row0 + row) * g.cap + F] = x;
    }
}

// ------------------------------------------------------------------ select
//
// One warp per row solves its threshold; every selected block sets its bit in the tile's bitmap
// (a ballot over the lanes is one word).  The CTA that finishes a tile turns the bitmap into
// the tile's list: selected full blocks ascending, the open block when it holds cached tokens
// (whether past or own), the tree itself last.
constexpr int kTreeSelWarps = 8;

__global__ void __launch_bounds__(kTreeSelWarps * 32)
tree_select_kernel(const int* __restrict__ kv_len, const int* __restrict__ n_nodes, const float* __restrict__ xs,
                   const unsigned long long* __restrict__ anc, const int* __restrict__ depth, float* __restrict__ tau,
                   unsigned* __restrict__ bits, int* __restrict__ tick, int* __restrict__ list, int* __restrict__ count,
                   int* __restrict__ offs, int* __restrict__ plan, __nv_bfloat16* __restrict__ out,
                   WsHeader* __restrict__ hdr, TreeGeom g, float alpha, int nctas, int per) {
    __shared__ int last_sh, wtot[kTreeSelWarps];
    constexpr int kCtasPerTile = kTreeRows / kTreeSelWarps;
    const int tile = blockIdx.x / kCtasPerTile, sub = blockIdx.x % kCtasPerTile;
    const int bg = tile / g.tiles_bg, b = bg / g.Hkv;
    const int r0 = (tile % g.tiles_bg) * kTreeRows, rows = min(kTreeRows, g.R - r0);
    if (sub * kTreeSelWarps >= rows) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int L, nodes;
    const bool live = tree_live(kv_len, n_nodes, g, b, &L, &nodes);
    const int F = live ? L / kBlock : 0, r = live ? L % kBlock : 0;
    const int lrow = sub * kTreeSelWarps + warp;                     // row of the tile
    if (lrow < rows) {
        const size_t row = (size_t)bg * g.R + r0 + lrow;
        const int node = (r0 + lrow) % g.N;
        const int dp = depth[(size_t)b * g.N + node];
        if (node < (n_nodes ? min(n_nodes[b], g.N) : g.N) && (!live || dp < 0)) {
            // no valid length or parent: zero output
            for (int c = lane; c < g.d; c += 32) out[row * g.d + c] = __float2bfloat16(0.f);
        }
        float t = __int_as_float(0x7fc00000);
        if (live && dp >= 0) {
            const int n = F + (r + dp >= kBlock ? 1 : 0);
            WarpRow xr;
            xr.load(xs + row * g.cap, lane, n);
            float m = -INFINITY;
            xr.each([&](int, float v) { m = fmaxf(m, v); });
            m = warp_max(m);
            int no_conv = 0;
            if (m > -INFINITY)
                t = alpha == 1.5f ? warp_row_tau<1>(xr, m, alpha, &no_conv, nullptr, g.maxit)
                  : alpha == 2.0f ? warp_row_tau<2>(xr, m, alpha, &no_conv, nullptr, g.maxit)
                                  : warp_row_tau<0>(xr, m, alpha, &no_conv, nullptr, g.maxit);
            if (no_conv && lane == 0) atomicOr(&hdr->status, kStNoConverge);
            int nsel = 0;
            const int words = (n + 31) / 32;
            auto word = [&](int k, float v) {
                const unsigned w = __ballot_sync(0xffffffffu, v > t);
                nsel += __popc(w);
                if (w && lane == 0) atomicOr(&bits[(size_t)tile * g.nbw + k], w);
            };
#pragma unroll
            for (int k = 0; k < kSelRegs; ++k)
                if (k < words) word(k, xr.r[k]);
            for (int k = kSelRegs; k < words; ++k) word(k, lane + 32 * k < n ? xr.p[lane + 32 * k] : -INFINITY);
            if (lane == 0) {
                atomicAdd(&hdr->selected_pairs, (unsigned long long)nsel);
                atomicAdd(&hdr->scored_pairs, (unsigned long long)n);
            }
        }
        if (lane == 0) tau[row] = t;
    }
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        last_sh = atomicAdd(&tick[tile], 1) == (rows + kTreeSelWarps - 1) / kTreeSelWarps - 1;
    }
    __syncthreads();
    if (!last_sh) return;
    __threadfence();
    int* dst = list + (size_t)tile * g.lcap;
    int total = 0;
    if (live) {
        const int nw = (F + 31) / 32;
        for (int w0 = 0; w0 < nw; w0 += kTreeSelWarps * 32) {
            const int wi = w0 + tid;
            unsigned word = wi < nw ? __ldcg(bits + (size_t)tile * g.nbw + wi) : 0u;
            if (wi == F / 32) word &= (1u << (F & 31)) - 1u;         // the open block has its own entry
            const int pc = __popc(word);
            int incl = pc;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) wtot[warp] = incl;
            __syncthreads();
            int pos = total + incl - pc;
            for (int w = 0; w < kTreeSelWarps; ++w) {
                if (w < warp) pos += wtot[w];
                total += wtot[w];
            }
            while (word) {
                dst[pos++] = wi * 32 + __ffs(word) - 1;
                word &= word - 1;
            }
            __syncthreads();
        }
        if (tid == 0) {
            atomicAdd(&hdr->union_blocks, (unsigned long long)total);
            if (total > 0) atomicAdd(&hdr->tiles, 1ull);
            if (r > 0) dst[total++] = kTreeOpen;
            dst[total++] = kTreeDraft;
        }
    }
    if (tid == 0) count[tile] = total;
    decode_plan_tail(count, offs, plan, hdr, g.tiles, nctas, per);
}

// ------------------------------------------------------------------ host side

constexpr int kTreePer = 4;          // list entries per CTA at least

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
    const auto* q = static_cast<const __nv_bfloat16*>(a.q);
    const auto* kd = static_cast<const __nv_bfloat16*>(a.k_draft);
    const auto* ks = static_cast<const uint8_t*>(a.k_scale);
    auto* out = static_cast<__nv_bfloat16*>(a.out);
    const dim3 gs((unsigned)(g.B * g.Hkv), (unsigned)((g.nbs + 63) / 64 + 1));
    const int nctas = tree_ctas();
    tree_scores_kernel<D, Q8><<<gs, 128, 0, stream>>>(q, kd, a.parent, a.n_nodes, a.k_cache, ks, a.ksum, a.kv_len, w.xs, w.anc,
                                                      w.depth, w.bits, w.tick, g, cx);
    tree_select_kernel<<<(unsigned)g.tiles * (kTreeRows / kTreeSelWarps), kTreeSelWarps * 32, 0, stream>>>(
        a.kv_len, a.n_nodes, w.xs, w.anc, w.depth, w.tau, w.bits, w.tick, w.list, w.count, w.offs, w.plan, out, w.hdr, g, alpha,
        nctas, kTreePer);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_tree_attn(a, w, g, e_pow, sm2, nctas, kTreePer, stream);
}

cudaError_t launch_tree(const TreeArgs& a, const TreeGeom& g, char* ws, float alpha, float coarse_scale, cudaStream_t stream) {
    if (g.d == 128) return a.k_scale ? launch_tree_t<128, true>(a, g, ws, alpha, coarse_scale, stream)
                                     : launch_tree_t<128, false>(a, g, ws, alpha, coarse_scale, stream);
    return a.k_scale ? launch_tree_t<64, true>(a, g, ws, alpha, coarse_scale, stream)
                     : launch_tree_t<64, false>(a, g, ws, alpha, coarse_scale, stream);
}

}  // namespace dash
