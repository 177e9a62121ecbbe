// tree.cuh -- what the kernels of a drafted-tree decode step share (tree.cu, tree_tc.cu).
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace dash {

constexpr int kTreeOpen = -1, kTreeDraft = -2;   // list entries behind the past blocks

// The workspace's regions.
struct TreeWork {
    WsHeader* hdr;
    float *xs, *tau;                     // scores [rows][cap], thresholds
    unsigned long long* anc;             // [B][N] ancestors and self (0: an invalid node)
    int* depth;                          // [B][N]
    float* path;                         // [B Hkv][N][D] 1 / 64 of the open block's keys on a node's path, added up
    unsigned* bits;                      // [tile][nbw] selected blocks
    int *tick, *list, *count;
    int* offs;                           // [tile] first entry of split tiles; [tiles]: entries in all
    float* part;                         // [CTA + tile] partials of 128 rows (tree_tc.cu)
};

inline TreeWork tree_work(const TreeGeom& g, char* ws) {
    TreeWork w;
    w.hdr = reinterpret_cast<WsHeader*>(ws);
    w.xs = reinterpret_cast<float*>(ws + g.off_x);
    w.tau = reinterpret_cast<float*>(ws + g.off_tau);
    w.anc = reinterpret_cast<unsigned long long*>(ws + g.off_anc);
    w.depth = reinterpret_cast<int*>(ws + g.off_depth);
    w.path = reinterpret_cast<float*>(ws + g.off_path);
    w.bits = reinterpret_cast<unsigned*>(ws + g.off_bits);
    w.tick = reinterpret_cast<int*>(ws + g.off_tick);
    w.list = reinterpret_cast<int*>(ws + g.off_list);
    w.count = reinterpret_cast<int*>(ws + g.off_count);
    w.offs = reinterpret_cast<int*>(ws + g.off_offs);
    w.part = reinterpret_cast<float*>(ws + g.off_part);
    return w;
}

// Whether the sequence's length is valid, and how many of its nodes are computed.
__device__ __forceinline__ bool tree_live(const int* kv_len, const int* n_nodes, const TreeGeom& g, int b, int* L, int* nodes) {
    *L = kv_len[b];
    *nodes = n_nodes ? max(0, min(n_nodes[b], g.N)) : g.N;
    return *L >= 0 && *L <= g.Tmax && *nodes > 0;
}

// attention over the tiles' lists on at most nctas CTAs, and the merge
cudaError_t launch_tree_attn(const TreeArgs& a, const TreeWork& w, const TreeGeom& g, float e_pow, float sm2, int nctas,
                             cudaStream_t stream);

}  // namespace dash
