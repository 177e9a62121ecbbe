// select.cuh -- threshold solves with one warp per row, and the work plan of the balanced
// split-KV pass: shared by the decode steps (decode.cu, tree.cu).
#pragma once

#include "common.cuh"
#include "entmax.cuh"

namespace dash {

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}
// all of the thread's cp.async copies have landed; no access moves across it
__device__ __forceinline__ void cp_async_done() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

// Shared memory of a decode step's select CTA for the rows it holds at a time (up to 8, one per warp): as many
// values of each as fit, and the rest from memory in every pass.  It is shared out over the rows there are: one
// head a group at 262,144 tokens needs 16 KB, not room for 8 rows, and several CTAs fit an SM (40 sequences of 8
// groups: 593 us a step against 655).  This is what an SM has beside the kernel's own 13 KB; at 1,048,576
// tokens, 4 heads, 4 sequences of 2 groups, a step takes 421 us with 24 KB, 364 with 96, 336 with 128 and 272
// with this (237 with passes over eight values at a time in place of four).
constexpr int kSelBytes = 208 * 1024;

// Row values a warp of a tree step's select CTA keeps in shared memory at most (128 KB for its 8 rows; shorter
// rows take less).  With 1536 a step at 262,144 tokens reads the rest from memory in every pass: a tree of 16
// over 2 KV heads takes 172 us, and 115 with 4096.
constexpr int kSelCap = 4096;

// Row values of one row on one warp, in shared memory: lane l holds x[l + 32 k]; values past the
// buffer are read from memory.  The buffer holds a multiple of 32 values, or the whole row.
struct WarpRow {
    const float *s, *p;
    int lane, n, ns;
    // buf: cap floats of this warp
    __device__ __forceinline__ void load(const float* row, float* buf, int cap, int ln, int count) {
        s = buf; p = row; lane = ln; n = count; ns = min(n, cap);
        if (((reinterpret_cast<size_t>(row) & 15) | (cap & 3)) == 0) {
            // whole chunks: up to 3 values past n, which no pass reads
            for (int j = 4 * lane; j < ns; j += 128) cp_async16(buf + j, row + j, 16);
        } else {
            for (int j = lane; j < ns; j += 32) cp_async4(buf + j, row + j);
        }
        cp_async_done();
        __syncwarp();
    }
    template <class F>
    __device__ __forceinline__ void each(F&& f) const {
        int j = lane;
#pragma unroll 8
        for (; j < ns; j += 32) f(j, s[j]);
#pragma unroll 8
        for (; j < n; j += 32) f(j, p[j]);
    }
    // largest of the lane's values
    __device__ __forceinline__ float lane_max() const {
        float m = -INFINITY;
        each([&](int, float v) { m = fmaxf(m, v); });
        return m;
    }
    // Bitmap of the values above t: calls f(k, word) for every word k with a bit set, on the lane
    // that holds it (a ballot over the lanes is a word; 32 words are gathered before their lanes
    // act, so that no word waits for the one before).  Returns the number of bits; every lane
    // calls it.
    template <class F>
    __device__ __forceinline__ int words(float t, F&& f) const {
        int bits = 0;
        for (int k0 = 0; k0 * 32 < n; k0 += 32) {
            const int kn = min(32, (n - k0 * 32 + 31) / 32);
            unsigned mine = 0u;
            const int ks = max(0, min(kn, (ns + 31) / 32 - k0));         // words whose values are in the buffer
#pragma unroll 8
            for (int k = 0; k < ks; ++k) {
                const int j = (k0 + k) * 32 + lane;
                const unsigned w = __ballot_sync(0xffffffffu, (j < ns ? s[j] : -INFINITY) > t);
                mine = lane == k ? w : mine;
            }
            // the others eight at a time: a load behind each ballot would wait for memory once a word
            for (int k = ks; k < kn; k += 8) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = p[min((k0 + k + i) * 32 + lane, n - 1)];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const unsigned w = __ballot_sync(0xffffffffu, (k0 + k + i) * 32 + lane < n && v[i] > t);
                    mine = lane == k + i ? w : mine;                     // 0 from word kn on
                }
            }
            bits += __popc(mine);
            if (mine) f(k0 + lane, mine);
        }
        return warp_sum_int(bits);
    }
};

// Turns a bitmap of nw words into the ascending list of its bits at dst, by all warps of the CTA
// (nwarp warps): a scan places the words, then a lane writes a bit.  word(i): word i; returns the
// number of bits.  sh: 33 nwarp ints of shared memory.
template <class W>
__device__ __forceinline__ int bits_to_list(const W& word, int nw, int* dst, int* sh, int nwarp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* wtot = sh;
    int* place = sh + nwarp;
    int total = 0;
    for (int w0 = 0; w0 < nw; w0 += nwarp * 32) {
        const int wi = w0 + tid;
        const int pc = wi < nw ? __popc(word(wi)) : 0;
        int incl = pc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) wtot[warp] = incl;
        __syncthreads();
        int pos = total + incl - pc;
        for (int k = 0; k < nwarp; ++k) {
            if (k < warp) pos += wtot[k];
            total += wtot[k];
        }
        place[tid] = pos;
        __syncthreads();
        const int nb = min(nwarp * 32, nw - w0);
        for (int k = warp; k < nb; k += nwarp) {
            const unsigned w = word(w0 + k);
            if ((w >> lane) & 1u) dst[place[k] + __popc(w & ((1u << lane) - 1u))] = (w0 + k) * 32 + lane;
        }
        __syncthreads();
    }
    return total;
}

constexpr int kHistBins = 64;       // bins of the histogram start over y = x - m in [-1, 0)

// Histogram start of the threshold solve (the idea of AdaSplash-2, whose abstract appears on
// the listing page "DashAttention: Differentiable and Adaptive Sparse Hierarchical Attention":
// a coarse histogram of the scores kept in on-chip memory gives a close initial threshold;
// the construction here is this library's):
// the values y = x - m in [-1, 0) go to bin k = floor((y + 1) * 64) with their count, sum and
// sum of squares, accumulated as integers (y and y^2 in 2^-24 fixed point), so the sums and
// the start do not depend on the order of the shared-memory atomics.  At a bin's lower edge
// e every value of the bins above lies above e, so f(e) = sum_{y > e} (y - e)^(1/(alpha-1))
// is exact there for alpha = 1.5 (S2 - 2 e S1 + e^2 S0) and alpha = 2 (S1 - e S0).  f is
// decreasing, so the highest edge with f >= 1 lies just below the root: Newton starts there
// instead of at -1.
// bins: this warp's shared area (kHistBins counts, then kHistBins sums, kHistBins sums of
// squares).  Every lane returns the start.
struct HistBins {
    unsigned int c[kHistBins];
    unsigned long long s1[kHistBins], s2[kHistBins];
};

template <int MODE>
__device__ __forceinline__ float hist_start(const WarpRow& xr, float m, HistBins* hb) {
    const int lane = threadIdx.x & 31;
    constexpr float kFix = 16777216.0f;                 // 2^24
    for (int i = lane; i < kHistBins; i += 32) { hb->c[i] = 0u; hb->s1[i] = 0ull; hb->s2[i] = 0ull; }
    __syncwarp();
    xr.each([&](int, float v) {
        const float y = v - m;
        if (y > -1.0f) {
            const int k = min(kHistBins - 1, (int)((y + 1.0f) * (float)kHistBins));
            atomicAdd(&hb->c[k], 1u);
            atomicAdd(&hb->s1[k], (unsigned long long)__float2ll_rn(y * kFix));
            atomicAdd(&hb->s2[k], (unsigned long long)__float2ll_rn(y * y * kFix));
        }
    });
    __syncwarp();
    // lane l holds bins 2l, 2l + 1; exact suffix sums over the bins at and above each edge
    long long c0 = hb->c[2 * lane], c1 = hb->c[2 * lane + 1];
    long long p0 = (long long)hb->s1[2 * lane], p1 = (long long)hb->s1[2 * lane + 1];
    long long q0 = (long long)hb->s2[2 * lane], q1 = (long long)hb->s2[2 * lane + 1];
    long long ac = c0 + c1, a1 = p0 + p1, a2 = q0 + q1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long nc = __shfl_down_sync(0xffffffffu, ac, o);
        const long long n1 = __shfl_down_sync(0xffffffffu, a1, o);
        const long long n2 = __shfl_down_sync(0xffffffffu, a2, o);
        if (lane + o < 32) { ac += nc; a1 += n1; a2 += n2; }
    }
    auto f_at = [&](int k, long long S0, long long S1q, long long S2q) {
        const double e = -1.0 + (double)k / kHistBins;
        const double S1 = (double)S1q / kFix, S2 = (double)S2q / kFix;
        return MODE == 1 ? S2 - 2.0 * e * S1 + e * e * (double)S0 : S1 - e * (double)S0;
    };
    const unsigned ok_odd = __ballot_sync(0xffffffffu, f_at(2 * lane + 1, ac - c0, a1 - p0, a2 - q0) >= 1.0);
    const unsigned ok_even = __ballot_sync(0xffffffffu, f_at(2 * lane, ac, a1, a2) >= 1.0);
    const int k_odd = ok_odd ? 2 * (31 - __clz((int)ok_odd)) + 1 : -1;
    const int k_even = ok_even ? 2 * (31 - __clz((int)ok_even)) : 0;
    __syncwarp();
    return -1.0f + (float)max(k_odd, k_even) / (float)kHistBins;
}

// Threshold of one row held by a warp (every lane returns it); MODE as in EntmaxPass::add_t.
// bins != nullptr: start from the histogram edge (alpha = 1.5 and 2), else from u = -1.
template <int MODE>
__device__ __forceinline__ float warp_row_tau(const WarpRow& xr, float m, float alpha, int* no_conv,
                                              HistBins* bins, int cap, float u0 = -1.0f) {
    if constexpr (MODE != 0) {
        if (bins) u0 = hist_start<MODE>(xr, m, bins);
    }
    EntmaxSolver sv;
    sv.init(m, alpha, u0, cap);
    float t = m;
    while (true) {
        EntmaxPass ps;
        ps.reset();
        xr.each([&](int, float v) { ps.add_t<MODE>((v - sv.m) - sv.u, sv.e); });
        ps.warp_reduce_t<MODE>();
        if (sv.update(ps, &t, no_conv)) break;
    }
    return t;
}

// Whether a query holds an element that is no finite number (one warp, every lane returns it).  Its row is NaN by
// its logits; a score of such a row that is infinite, or none that is a number, is no failed solve.  Not inlined:
// in line, this rare code takes the decode select pass from 64 registers to 104 and a step of 4 x 1M tokens from 242 us to 266.
static __device__ __noinline__ bool row_not_finite(const __nv_bfloat16* q, int d) {
    bool bad = false;
    for (int c = threadIdx.x & 31; c < d; c += 32) bad |= !(fabsf(__bfloat162float(q[c])) < INFINITY);
    return __any_sync(0xffffffffu, bad);
}

// The threshold of a row whatever alpha is; m = its largest value, finite.
__device__ __forceinline__ float row_tau(const WarpRow& xr, float m, float alpha, int* no_conv, HistBins* bins,
                                         int cap, float u0 = -1.0f) {
    return alpha == 1.5f ? warp_row_tau<1>(xr, m, alpha, no_conv, bins, cap, u0)
         : alpha == 2.0f ? warp_row_tau<2>(xr, m, alpha, no_conv, bins, cap, u0)
                         : warp_row_tau<0>(xr, m, alpha, no_conv, bins, cap, u0);
}

// A start below the root from the lanes' 32 largest values (a subset's root never exceeds the
// row's, entmax.cuh): one value per lane, so its passes cost a reduction each, and a few passes
// over the row are left of the eight or so from u = -1.
template <int MODE>
__device__ __forceinline__ float lane_start_t(float y, float alpha) {
    EntmaxSolver sv;
    sv.init(0.0f, alpha);
    float t = -1.0f;
    int nc = 0;
    for (int it = 0; it < 24; ++it) {
        EntmaxPass ps;
        ps.reset();
        ps.add_t<MODE>(y - sv.u, sv.e);
        ps.warp_reduce_t<MODE>();
        if (sv.update(ps, &t, &nc)) return (nc || !(t >= -1.0f)) ? sv.lo : fminf(t, -1e-30f);
    }
    return sv.lo;
}
// y: the lane's largest value less the row's
__device__ __forceinline__ float lane_start(float y, float alpha) {
    return alpha == 1.5f ? lane_start_t<1>(y, alpha) : alpha == 2.0f ? lane_start_t<2>(y, alpha) : lane_start_t<0>(y, alpha);
}

// CTAs that share the U entries of `lists` lists: at most `grid`, and no more than pay.  p CTAs on a list of
// e entries take e / p entries' time, and its merge p pieces'; with an entry as long as `ratio` pieces,
// p = sqrt(e ratio), or sqrt(e / ratio) entries a CTA.  ratio 0: pieces cost nothing to speak of.
__device__ __forceinline__ int split_ctas(int U, int lists, int grid, int ratio) {
    const unsigned per = ratio > 0 ? (unsigned)fmaxf(1.0f, sqrtf((float)U / ((float)lists * (float)ratio))) : 1u;
    const unsigned n = ((unsigned)U + per - 1u) / per;
    return n < (unsigned)grid ? (int)n : grid;
}

// The ranges [U c / n, U (c + 1) / n) of the n CTAs that share U > 0 entries, in 32-bit arithmetic
// (n <= kDecodeMaxCtas; a 64-bit division costs a few hundred cycles where a step has none to lose).
struct ListSplit {
    unsigned U, n, q, r;
    __device__ __forceinline__ ListSplit(int U_, int lists, int grid, int ratio)
        : U((unsigned)U_), n((unsigned)split_ctas(U_, lists, grid, ratio)) {
        q = n ? U / n : 0u;
        r = U - q * n;
    }
    __device__ __forceinline__ int lo(int c) const { return (int)(q * (unsigned)c + (n ? r * (unsigned)c / n : 0u)); }
    // the CTA whose range holds position pos: an estimate (relative error below 2^-21, so at most one
    // off), put right
    __device__ __forceinline__ int cta_of(int pos) const {
        int c = min((int)n - 1, (int)((float)pos / (float)U * (float)n));
        while (c > 0 && lo(c) > pos) --c;
        while (c + 1 < (int)n && lo(c + 1) <= pos) ++c;
        return c;
    }
};

// CTA c's range and the number of CTAs.  Not inlined: in line, its divisions cost the attention kernels
// registers to the end (240 bytes of spills a thread in the 8-bit tree variant).
static __device__ __noinline__ int3 cta_range(int U, int lists, int grid, int ratio, int c) {
    const ListSplit sp(U, lists, grid, ratio);
    return make_int3(sp.lo(c), sp.lo(c + 1), (int)sp.n);
}

// Where list x lies in the concatenation: its first entry, its length, and the entries of all.  A merge
// that starts before the attention has ended adds up the lists' lengths itself, so that nothing is
// left to look up when it ends (16K tree: 14 us of merge, 4 with this and its loads together); from
// kPlaceLists lists on, where every CTA's sums would weigh more, it takes what the attention leaves in
// offs ([x] first entry, [lists] entries in all).  All NT threads of the CTA call it; sh: NT / 16 ints.
constexpr int kPlaceLists = 1024;
struct ListPlace {
    int U, o0, n;
};
__device__ __forceinline__ void pdl_wait();
template <int NT>
__device__ __forceinline__ ListPlace list_place(const int* count, const int* offs, int lists, int x, int* sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (lists >= kPlaceLists) {
        pdl_wait();
        return ListPlace{__ldcg(offs + lists), __ldcg(offs + x), __ldcg(count + x)};
    }
    int all = 0, before = 0;
    for (int i = tid; i < lists; i += NT) {
        const int c = __ldcg(count + i);
        all += c;
        before += i < x ? c : 0;
    }
    ListPlace r;
    r.n = __ldcg(count + x);
    all = warp_sum_int(all);
    before = warp_sum_int(before);
    if (lane == 0) { sh[warp] = all; sh[NT / 32 + warp] = before; }
    __syncthreads();
    r.U = r.o0 = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) { r.U += sh[w]; r.o0 += sh[NT / 32 + w]; }
    return r;
}

// A CTA's share of the concatenated lists, from their lengths alone: U entries in all, nC CTAs
// with work, entries [lo, hi) for this one (empty for a CTA past nC), which begin in list
// `first`, whose own entries are [o_first, o_end).  All NT threads of the CTA call it; sh: NT / 32 + 3 ints.
struct ListShare {
    int U, nC, lo, hi, first, o_first, o_end;
};
template <int NT>
__device__ __forceinline__ ListShare list_share(const int* count, int lists, int cta, int grid, int ratio, int* sh) {
    constexpr int KEEP = 4;                            // lengths a thread keeps
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = (lists + NT - 1) / NT, i0 = min(lists, tid * chunk), i1 = min(lists, i0 + chunk);
    int c[KEEP], sum = 0;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) c[k] = i0 + k < i1 ? __ldcg(count + i0 + k) : 0;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) sum += c[k];
    for (int i = i0 + KEEP; i < i1; ++i) sum += __ldcg(count + i);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    int pre = incl - sum;
    ListShare r;
    r.U = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) pre += sh[w];
        r.U += sh[w];
    }
    const int3 range = cta_range(r.U, lists, grid, ratio, cta);
    r.nC = range.z;
    r.lo = r.hi = 0;
    if (cta < r.nC) {
        r.lo = range.x;
        r.hi = range.y;
    }
    if (r.lo < r.hi && r.lo >= pre && r.lo < pre + sum) {
        // one thread's lists hold the first entry
        int i = i0, o = pre, n = 0;
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (i == i0 + k && i < i1) {
                n = c[k];
                if (o + n <= r.lo) { o += n; ++i; }
            }
        for (; i >= i0 + KEEP && (n = __ldcg(count + i), o + n <= r.lo); ++i) o += n;
        sh[NT / 32] = i;
        sh[NT / 32 + 1] = o;
        sh[NT / 32 + 2] = o + n;
    }
    __syncthreads();
    r.first = sh[NT / 32];
    r.o_first = sh[NT / 32 + 1];
    r.o_end = sh[NT / 32 + 2];
    return r;
}

// A warp's walk along list entries [e, end): 64 of them in registers, so that a producer neither
// waits for one entry's load before each copy nor reads ahead one by one.  at(e + k) for
// k < 32 from the current entry e; every lane calls it.
struct ListWindow {
    const int* p;
    int base, end, cur, nxt;
    __device__ __forceinline__ int fetch(int e) const {
        const int i = e + (threadIdx.x & 31);
        return i < end ? __ldcg(p + i) : 0;
    }
    __device__ __forceinline__ void start(const int* list, int e, int e_end) {
        p = list; base = e; end = e_end;
        cur = fetch(e);
        nxt = fetch(e + 32);
    }
    // the entry is now e (called with e increasing by one)
    __device__ __forceinline__ void to(int e) {
        if (e - base == 32) {
            base = e;
            cur = nxt;
            nxt = fetch(e + 32);
        }
    }
    __device__ __forceinline__ int at(int e) const {
        const int k = e - base;
        return __shfl_sync(0xffffffffu, k < 32 ? cur : nxt, k & 31);
    }
};

// Programmatic dependent launch: a kernel that calls pdl_trigger lets its successor's blocks start
// (launched with PdlConfig) and run up to pdl_wait, which returns once every kernel before it
// has finished and its writes are visible.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct PdlConfig {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    PdlConfig(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) : cfg{} {
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

// Work plan of the balanced attention pass, built by the last select CTA to finish (a
// ticket in the workspace header): offs = exclusive prefix of the list lengths (U = offs[BH]
// blocks in all), and plan[c] = the group holding position floor(U c / n), where CTA c's
// range starts (n = min(nctas, U)).  Called by every thread of every CTA once its count is
// written.
static __device__ void decode_plan_tail(const int* count, int* offs, int* plan, WsHeader* hdr, int BH, int nctas) {
    __shared__ int last_sh;
    __shared__ int wsum[32];
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();                              // this CTA's count before its ticket
        last_sh = atomicAdd(&hdr->ticket, 1) == BH - 1;
    }
    __syncthreads();
    if (!last_sh) return;
    __threadfence();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
    const int slice = (BH + nwarp - 1) / nwarp;
    const int lo = min(BH, warp * slice), hi = min(BH, lo + slice);
    int sum = 0;
    for (int i = lo + lane; i < hi; i += 32) sum += __ldcg(count + i);
    sum = warp_sum_int(sum);
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
    int before = 0, U = 0;
    for (int w = 0; w < nwarp; ++w) {
        if (w < warp) before += wsum[w];
        U += wsum[w];
    }
    if (threadIdx.x == 0) offs[BH] = U;
    nctas = min(U, nctas);                            // the attention pass uses min(grid, U) CTAs
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const int v = i < hi ? __ldcg(count + i) : 0;
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        const int o0 = before + incl - v, o1 = before + incl;
        if (i < hi) {
            offs[i] = o0;
            if (v > 0) {
                // CTAs whose range starts inside [o0, o1)
                const int c_lo = (int)(((long long)o0 * nctas + U - 1) / U);
                const int c_hi = (int)(((long long)o1 * nctas - 1) / U);
                for (int c = c_lo; c <= c_hi; ++c) plan[c] = i;
            }
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

}  // namespace dash
