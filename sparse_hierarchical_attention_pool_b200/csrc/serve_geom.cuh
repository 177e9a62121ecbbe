// serve_geom.cuh -- workspace layouts of the decode steps over the 8-bit KV cache and over drafted-token trees.
#pragma once

#include "common.cuh"

namespace dash {

// Geometry of a decode step over the 8-bit cache.  Its attention kernel takes at most 8 heads
// (one n8 tile), so a KV group of more heads becomes `split` virtual groups of G / split heads,
// each with its own block list (split = the least divisor of G with G / split <= 8).  Scores
// need the real groups, lists and attention the virtual ones; both share the score and
// threshold rows of the workspace, whose offsets depend on Hq and Tmax alone.
struct DecodeQ8Geom {
    DecodeGeom real, v;
    int split;
};

inline bool make_decode_q8_geom(int B, int Hq, int Hkv, int Tmax, int d, DecodeQ8Geom* g) {
    if (!make_decode_geom(B, Hq, Hkv, Tmax, d, &g->real) || Tmax % kBlock != 0) return false;
    if ((long long)B * Hkv * Tmax >= (1ll << 31)) return false;
    g->split = 1;
    while (g->real.G % g->split != 0 || g->real.G / g->split > 8) ++g->split;
    if (!make_decode_geom(B, Hq, Hkv * g->split, Tmax, d, &g->v)) return false;
    // partials hold two maxima and the sum (16 bytes with padding) and the output per head
    const size_t slots = ((size_t)B * Hkv * g->split + kDecodeMaxCtas) * 4;      // one per consumer warp
    g->v.total = align256(g->v.off_part + slots * g->v.G * (d + 4) * sizeof(float));
    return true;
}

// Geometry of a decode step over drafted-token trees: the rows of a KV group are its G heads x
// N nodes (r = head_local * N + node, contiguous rows of q), cut into tiles of kTreeRows.
constexpr int kMaxNodes = 64;        // nodes per tree: an ancestor set is one 64-bit mask
constexpr int kTreeRows = 128;       // rows of a tile

struct TreeGeom {
    int B, Hq, Hkv, N, Tmax, d, G, nbs;
    int R;                           // rows per KV group = G * N
    int tiles_bg, tiles;             // tiles per KV group, in all
    int cap;                         // scores per row: the full blocks and the open one, and padding
    int lcap;                        // list entries per tile: the full blocks, the open one, the tree
    int nbw;                         // 32-bit words of a tile's selection bitmap
    int maxit;
    size_t off_x, off_tau, off_anc, off_depth, off_path, off_bits, off_tick, off_list, off_count, off_offs, off_part,
        total;
};

inline bool make_tree_geom(int B, int Hq, int Hkv, int N, int Tmax, int d, TreeGeom* g) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Tmax < 1 || Tmax > kMaxT || (Hq % Hkv) != 0) return false;
    if ((d != 64 && d != 128) || N < 1 || N > kMaxNodes || Hq / Hkv > 32) return false;
    if ((long long)B * Hkv * Tmax >= (1ll << 31) || (long long)B * Hq * N >= (1ll << 31)) return false;
    g->B = B; g->Hq = Hq; g->Hkv = Hkv; g->N = N; g->Tmax = Tmax; g->d = d; g->G = Hq / Hkv;
    g->nbs = Tmax / kBlock;
    g->R = g->G * N;
    g->tiles_bg = (g->R + kTreeRows - 1) / kTreeRows;
    g->tiles = B * Hkv * g->tiles_bg;
    g->cap = (g->nbs + 4) & ~3;      // rows of scores begin on 16 bytes
    g->lcap = g->nbs + 2;
    g->nbw = (g->nbs + 32) / 32;
    g->maxit = solve_cap_from_env();
    const size_t rows = (size_t)B * Hq * N, tiles = (size_t)g->tiles;
    size_t off = align256(sizeof(WsHeader));
    g->off_x = off;     off = align256(off + rows * g->cap * sizeof(float));
    g->off_tau = off;   off = align256(off + rows * sizeof(float));
    g->off_anc = off;   off = align256(off + (size_t)B * N * sizeof(unsigned long long));
    g->off_depth = off; off = align256(off + (size_t)B * N * sizeof(int));
    g->off_path = off;  off = align256(off + (size_t)B * Hkv * N * d * sizeof(float));
    g->off_bits = off;  off = align256(off + tiles * g->nbw * sizeof(unsigned));
    g->off_tick = off;  off = align256(off + tiles * sizeof(int));
    g->off_list = off;  off = align256(off + tiles * g->lcap * sizeof(int));
    g->off_count = off; off = align256(off + tiles * sizeof(int));
    g->off_offs = off;  off = align256(off + (tiles + 1) * sizeof(int));
    // partial (max, sum, padding to 16 bytes, output) per row of a (CTA + tile) slot
    g->off_part = off;  off = align256(off + (tiles + kDecodeMaxCtas) * kTreeRows * (d + 4) * sizeof(float));
    g->total = off;
    return true;
}

}  // namespace dash
