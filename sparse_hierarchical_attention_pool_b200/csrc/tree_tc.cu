// tree_tc.cu -- attention of a drafted-tree decode step on tcgen05, split over the concatenated
// lists of the tiles (tree.cu: what a list holds).
//
// A tile is up to 128 rows (heads x nodes) of one KV group and the M rows of both products:
// S = Q K^T (N = 64 keys) into TMEM, softmax weights P back into TMEM, O += P V in TMEM.  The
// tensor core does 128 rows at the price of one, so rows that a tile lacks cost no time.  Q and P
// are A operands in TMEM: with both in shared memory its 128 bytes a cycle were what bounded
// a step (80 KB of operands and 48 KB of writes; now 32 KB and 32 KB), not HBM.
//
// Work split as in decode_q8.cu, but with as many CTAs as there are entries (an entry is 1.5 us of its CTA, a
// piece one more of the merge's loads that go out together; 2 x 0.9K, 5 nodes: 4 entries a CTA at least
// 26.7 us a step, 2 24.6, 1 20.6): the lists laid end to end hold U entries, CTA c of n takes entries
// [U c / n, U (c + 1) / n); a tile inside one CTA is finished there, the others leave
// (max, sum, output) per row in slot CTA + tile for tree_combine_kernel.
//
// Roles (warps): 0 - 7 softmax, two groups of 128 threads (one per row) that take the steps
// alternately, each with its own S, P, O, sum and maximum, merged at the end of a segment;
// 8 K producer; 9 issuer of S; 10 issuer of P V; 11 V producer.  Counters of rings and barriers
// run over the CTA's whole range; only Q and the accumulators belong to a segment.  The value rows
// that no row may attend (the open block's behind the sequence, the draft's behind its nodes)
// are zeros in the product: weight 0 times whatever they hold would not be 0 if that were NaN.
//
// 8-bit cache: warp 8 streams codes and scale bytes with bulk copies into a ring of their own, and
// warps 12 - 15 (K) and 16 - 19 (V) turn them into bf16 operand tiles (exact: cache8.cuh) or load
// the draft's bf16 rows.  Two warps a tensor convert too slowly (32K, 4 x 24 nodes: 112 us a step
// against 93), eight gain nothing; tiles of f16 codes with the scales outside the product save
// conversions but need another factor per step in every role, and measured 115.
//
// The row sums take the unrounded weights, the products weights of 8 bits (that rounding is what a step's error
// has beyond its bf16 output's: 0.0022 against 0.0017 in the 2-norm).  Summing the rounded ones, so that a
// row's add up to one exactly, costs two more instructions a pair in the softmax: 466 us a step against 314 (96K, as
// below), 112 against 92 (8-bit, 32K).
//
// bf16 cache: bound by HBM and the softmax's instructions alike; 96K, 8 sequences of 32 / 8 heads and 16 nodes:
// the listed blocks' 1.71 GB in 263 us, 6.5 TB/s, at 1965 MHz.  Steps that follow one another draw the card's 1000 W
// within a second; at the 1550 MHz that its power cap leaves then, a whole step takes 355 us and not 316.
// 8-bit cache: bound by the roles' instructions; 32K, 4 sequences, 24 nodes: 45 entries
// a CTA in 55 to 62 us, 2,500 cycles each, of which the converters, which wait for nothing, need all.
// Every wait is bounded; a CTA that gives up sets a status bit.
#include "cache8.cuh"
#include "kernels.h"
#include "select.cuh"
#include "sm100.cuh"
#include "tree.cuh"

namespace dash {

constexpr int kTtRaw = 6;              // 8-bit ring
constexpr int kTtConv = 4;             // converter warps for K, and for V
template <bool Q8>
constexpr int kTtThreads = Q8 ? 384 + kTtConv * 64 : 384;
constexpr float kTtLazy = 8.0f;        // log2 units a maximum may grow before O is rescaled

template <int D, bool Q8>
struct TtLayout {
    static constexpr int kKS = Q8 ? 2 : 5, kVS = Q8 ? 3 : 5;    // operand tile rings
    static constexpr uint32_t kHalf = 64 * 128;                 // 64 rows x 64 elements
    static constexpr uint32_t kTile = (D / 64) * kHalf;         // K or V of one entry
    static constexpr uint32_t kRawKV = 64 * D;                  // codes of K or V of one entry
    static constexpr uint32_t kRaw = 2 * kRawKV + 128;          // and the scale bytes
    static constexpr uint32_t off_k = 0;
    static constexpr uint32_t off_v = off_k + kKS * kTile;
    static constexpr uint32_t off_raw = off_v + kVS * kTile;
    static constexpr uint32_t used = off_raw + (Q8 ? kTtRaw * kRaw : 0) + 1024;
    // more than half an SM's shared memory: the CTA's 512 TMEM columns are all there are
    static constexpr uint32_t bytes = used > 120 * 1024 ? used : 120 * 1024;
    static_assert(bytes + 4096 <= 227 * 1024, "shared memory of one CTA per SM");
    // TMEM columns: S of group g at 64 g, O at 128 + D g, Q (two 16-bit elements a column), P of group g
    static constexpr uint32_t colO = 128, colQ = 384, colP = 448;
};

// One 32-bit word of codes as four bf16, scaled: the code's exponent and mantissa bits moved to
// bf16's place read as code 2^-120 (subnormals too), so two exact multiplications by powers of
// two give code 2^(s - 127).  f2: 2^(s - 127) in both halves.
__device__ __forceinline__ void e4m3x4_to_bf16x4(uint32_t w, uint32_t f2, uint32_t* lo, uint32_t* hi) {
    const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(&f2);
    const __nv_bfloat162 up = __floats2bfloat162_rn(0x1p120f, 0x1p120f);
    const uint32_t e = __byte_perm(w, 0u, 0x1404), o = __byte_perm(w, 0u, 0x3424);   // codes 0, 1 and 2, 3 in the high bytes
    const uint32_t a = (e & 0x80008000u) | ((e >> 4) & 0x07f007f0u), b = (o & 0x80008000u) | ((o >> 4) & 0x07f007f0u);
    const __nv_bfloat162 x = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), up), f);
    const __nv_bfloat162 y = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), up), f);
    *lo = *reinterpret_cast<const uint32_t*>(&x);
    *hi = *reinterpret_cast<const uint32_t*>(&y);
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kTtThreads<Q8>, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_kd, const __grid_constant__ CUtensorMap tm_vd, TreeArgs a,
                 TreeWork w, TreeGeom g, float e_pow, float sm2) {
    using L = TtLayout<D, Q8>;
    using namespace sm100;
    constexpr int KS = L::kKS, VS = L::kVS;
    enum : int { B_Q = 0, B_KF = 1, B_KE = B_KF + KS, B_VF = B_KE + KS, B_VE = B_VF + VS, B_SF = B_VE + VS, B_SE = B_SF + 2,
                 B_PF = B_SE + 2, B_PD = B_PF + 2, B_RF = B_PD + 2, B_RE = B_RF + kTtRaw,
                 B_VT = B_RE + kTtRaw, B_DR = B_VT + 1, B_COUNT = B_DR + 2 };
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[B_COUNT];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    __shared__ float m_sh[2][kTreeRows], l_sh[2][kTreeRows];     // the groups' maxima and sums
    constexpr int NT = kTtThreads<Q8>;
    __shared__ int share_sh[NT / 32 + 3];
    const int cta = blockIdx.x;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const base_ptr = smem_raw + (base - raw);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const auto* q = static_cast<const __nv_bfloat16*>(a.q);
    if (tid == 0) {
        abort_sh = 0;
        const int conv = Q8 ? kTtConv : 1;                      // who fills an operand tile
        mbar_init(bar(B_Q), 4);
        for (int i = 0; i < KS; ++i) { mbar_init(bar(B_KF + i), conv); mbar_init(bar(B_KE + i), 1); }
        for (int i = 0; i < VS; ++i) { mbar_init(bar(B_VF + i), conv); mbar_init(bar(B_VE + i), 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_SF + i), 1);
            mbar_init(bar(B_SE + i), 4);
            mbar_init(bar(B_PF + i), 4);
            mbar_init(bar(B_PD + i), 1);
            mbar_init(bar(B_DR + i), 1);
        }
        for (int i = 0; i < kTtRaw; ++i) { mbar_init(bar(B_RF + i), 1); mbar_init(bar(B_RE + i), 2 * kTtConv); }
        mbar_init(bar(B_VT), 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_sh), 512);
        tmem_relinquish();
    }
    if constexpr (!Q8) {
        if (warp == 8 && lane == 0) { prefetch_tmap(&tm_k); prefetch_tmap(&tm_kd); }
        if (warp == 11 && lane == 0) { prefetch_tmap(&tm_v); prefetch_tmap(&tm_vd); }
    }
    tc_fence_before();
    pdl_wait();
    pdl_trigger();                                               // after the wait: the merge may read the lists at once
    // its barriers also publish the set-up above
    const ListShare sh = list_share<NT>(w.count, g.tiles, cta, (int)gridDim.x, 0, share_sh);
    tc_fence_after();
    if (cta == 0 && tid == 0) w.offs[g.tiles] = sh.U;
    const uint32_t tmem = tmem_sh;
    volatile int* abort_flag = &abort_sh;
    auto k_addr = [&](int st) { return base + L::off_k + (uint32_t)st * L::kTile; };
    auto v_addr = [&](int st) { return base + L::off_v + (uint32_t)st * L::kTile; };

    // one arrival a warp: 32 lanes' arrivals at one barrier are served one after another
    auto arrive = [&](uint32_t bar_addr) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_addr);
    };

    // calls body(tile, first entry, entries, steps before, the tile's first entry in the
    // concatenation, its end) for every segment of the range
    auto segments = [&](auto&& body) {
        int gs = 0;
        for (int tile = sh.first, pos = sh.lo, o0 = sh.o_first, o1; pos < sh.hi; ++tile, o0 = o1) {
            o1 = tile == sh.first ? sh.o_end : o0 + __ldcg(w.count + tile);
            if (o1 <= pos) continue;
            const int n = min(sh.hi, o1) - pos;
            body(tile, pos - o0, n, gs, o0, o1);
            pos += n;
            gs += n;
        }
    };

    // Q8: 640 threads have 96 registers each; the softmax's 64 scores a thread want more, the others less
    // (256 x 136 + 128 x 56 + 256 x 72 = 60,416 of the 61,440 the block holds)
    if (warp >= 8 && warp < 12) {
        if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");
    if (warp == 8) {
        // ------------------------------------------------------------ K producer / 8-bit stream
        // one lane copies, the warp walks the list
        bool ok = true;
        int armed = 0;                                           // steps loaded
        segments([&](int tile, int e0, int n, int gs, int, int) {
            const int bg = tile / g.tiles_bg;
            const int F = a.kv_len[bg / g.Hkv] / kBlock;
            ListWindow win;
            win.start(w.list + (size_t)tile * g.lcap, e0, e0 + n);
            for (int s = 0; ok && s < n; ++s) {
                win.to(e0 + s);
                const int j = win.at(e0 + s);
                if constexpr (Q8) {
                    if (j == kTreeDraft) continue;               // loaded by the converters
                    const int st = armed % kTtRaw;
                    const bool got = armed < kTtRaw || mbar_wait(bar(B_RE + st), ((armed / kTtRaw) - 1) & 1, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                    if (lane == 0) {
                        const size_t row = (size_t)bg * g.Tmax + (size_t)(j == kTreeOpen ? F : j) * kBlock;
                        const uint32_t dst = base + L::off_raw + (uint32_t)st * L::kRaw, bf = bar(B_RF + st);
                        mbar_arrive_expect_tx(bf, L::kRaw);
                        bulk_load_1d(dst, static_cast<const uint8_t*>(a.k_cache) + row * D, L::kRawKV, bf);
                        bulk_load_1d(dst + L::kRawKV, static_cast<const uint8_t*>(a.v_cache) + row * D, L::kRawKV, bf);
                        bulk_load_1d(dst + 2 * L::kRawKV, static_cast<const uint8_t*>(a.k_scale) + row, 64, bf);
                        bulk_load_1d(dst + 2 * L::kRawKV + 64, static_cast<const uint8_t*>(a.v_scale) + row, 64, bf);
                    }
                } else {
                    const int st = (gs + s) % KS;
                    const bool got = gs + s < KS || mbar_wait(bar(B_KE + st), (((gs + s) / KS) - 1) & 1, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(B_KF + st), L::kTile);
                        const CUtensorMap* tm = j == kTreeDraft ? &tm_kd : &tm_k;
                        const int row = j == kTreeDraft ? bg * g.N : bg * g.Tmax + (j == kTreeOpen ? F : j) * kBlock;
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) tma_load_2d(k_addr(st) + h * L::kHalf, tm, h * 64, row, bar(B_KF + st));
                    }
                }
                ++armed;
            }
        });
        if (lane == 0) {
            // every load this thread started lands before the CTA exits, also where another role gives up after the last
            constexpr int NS = Q8 ? kTtRaw : KS;
            volatile int dummy = 0;
            for (int st = 0; st < NS; ++st) {
                if (armed <= st) continue;
                const int last = armed - 1 - ((armed - 1 - st) % NS);
                dummy = 0;
                mbar_wait(bar((Q8 ? (int)B_RF : (int)B_KF) + st), (last / NS) & 1, &dummy);
            }
        }
    } else if (warp == 11) {
        // ------------------------------------------------------------ V producer (bf16 cache)
        if constexpr (!Q8) {
            bool ok = true;
            int special = 0, last_st[VS];
#pragma unroll
            for (int i = 0; i < VS; ++i) last_st[i] = -1;
            segments([&](int tile, int e0, int n, int gs, int, int) {
                const int bg = tile / g.tiles_bg, b = bg / g.Hkv;
                int len, nodes;
                tree_live(a.kv_len, a.n_nodes, g, b, &len, &nodes);
                const int F = len / kBlock;
                ListWindow win;
                win.start(w.list + (size_t)tile * g.lcap, e0, e0 + n);
                for (int s = 0; ok && s < n; ++s) {
                    win.to(e0 + s);
                    const int j = win.at(e0 + s);
                    const int st = (gs + s) % VS;
                    bool got = gs + s < VS || mbar_wait(bar(B_VE + st), (((gs + s) / VS) - 1) & 1, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                    const CUtensorMap* tm = j == kTreeDraft ? &tm_vd : &tm_v;
                    const int row = j == kTreeDraft ? bg * g.N : bg * g.Tmax + (j == kTreeOpen ? F : j) * kBlock;
                    const int bf = j < 0 ? (int)B_VT : (int)B_VF + st;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(bf), L::kTile);
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) tma_load_2d(v_addr(st) + h * L::kHalf, tm, h * 64, row, bar(bf));
                    }
                    if (j < 0) {
                        got = mbar_wait(bar(B_VT), special & 1, abort_flag);
                        ++special;
                        if (!__all_sync(0xffffffffu, got)) {
                            // the special load itself is still to land
                            volatile int dummy = 0;
                            if (!got) mbar_wait(bar(B_VT), (special - 1) & 1, &dummy);
                            ok = false;
                            break;
                        }
                        const int lim = j == kTreeDraft ? nodes : len % kBlock;
                        for (int i = lane; i < (kBlock - lim) * (D / 8); i += 32) {
                            const int r = lim + i / (D / 8), c = i % (D / 8);
                            *reinterpret_cast<uint4*>(base_ptr + L::off_v + st * L::kTile + (c >> 3) * L::kHalf + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_VF + st));
                    }
                    // the stage's last use, special entries too: an older one's parity would wait in vain
#pragma unroll
                    for (int i = 0; i < VS; ++i)
                        if (i == st) last_st[i] = gs + s;
                }
            });
            if (lane == 0) {
                volatile int dummy = 0;
#pragma unroll
                for (int i = 0; i < VS; ++i)
                    if (last_st[i] >= 0) { dummy = 0; mbar_wait(bar(B_VF + i), (last_st[i] / VS) & 1, &dummy); }
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------ S issuer
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16(128, 64, false);
            // descriptors are linear in the address (its bits fit the field)
            const uint64_t dk0 = smem_desc_sw128(base + L::off_k, 16, 1024);
            bool ok = true;
            int seg = 0;
            segments([&](int, int, int n, int gs0, int, int) {
                if (ok && !mbar_wait(bar(B_Q), seg & 1, abort_flag)) ok = false;
                ++seg;
                for (int s = 0; ok && s < n; ++s) {
                    const int gs = gs0 + s, st = gs % KS, sb = gs & 1, i2 = gs >> 1;
                    if (!mbar_wait(bar(B_KF + st), (gs / KS) & 1, abort_flag)) { ok = false; break; }
                    if (i2 >= 1 && !mbar_wait(bar(B_SE + sb), (i2 - 1) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t dk = dk0 + (uint32_t)st * (L::kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_bf16_ts(tmem + sb * 64, tmem + L::colQ + kk * 8, dk + (kk >> 2) * (L::kHalf >> 4) + (kk & 3) * 2, idesc, kk > 0 ? 1u : 0u);
                    mma_commit(bar(B_SF + sb));
                    mma_commit(bar(B_KE + st));
                }
            });
            if (!ok) {
                mma_commit(bar(B_DR));
                volatile int dummy = 0;
                mbar_wait(bar(B_DR), 0, &dummy);
            }
        }
    } else if (warp == 10) {
        // ------------------------------------------------------------ PV issuer
        if (lane == 0) {
            const uint32_t idesc_v = idesc_bf16(128, D, true);
            const uint64_t dv0 = smem_desc_sw128(base + L::off_v, L::kHalf, 1024);
            bool ok = true;
            segments([&](int, int, int n, int gs0, int, int) {
                for (int s = 0; ok && s < n; ++s) {
                    const int gs = gs0 + s, st = gs % VS, gp = gs & 1, i2 = gs >> 1;
                    if (!mbar_wait(bar(B_VF + st), (gs / VS) & 1, abort_flag)) { ok = false; break; }
                    if (!mbar_wait(bar(B_PF + gp), i2 & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t acc = s >= 2 ? 1u : 0u;       // a group's first step of the segment overwrites
                    const uint64_t dv = dv0 + (uint32_t)st * (L::kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ts(tmem + L::colO + gp * D, tmem + L::colP + gp * 32 + kk * 8, dv + kk * 128, idesc_v, (acc || kk > 0) ? 1u : 0u);
                    mma_commit(bar(B_PD + gp));
                    mma_commit(bar(B_VE + st));
                }
            });
            if (!ok) {
                mma_commit(bar(B_DR + 1));
                volatile int dummy = 0;
                mbar_wait(bar(B_DR + 1), 0, &dummy);
            }
        }
    }
    } else if (warp >= 12) {
        if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
        // ------------------------------------------------------------ converters (8-bit cache)
        if constexpr (Q8) {
            // warps for K and warps for V, each at its own ring's pace: V tiles are free only
            // after their product, K tiles long before
            constexpr int CH = D / 16;                           // 16-code chunks per row
            const int kv = (warp - 12) / kTtConv, ct = (tid - 384) % (kTtConv * 32), NS = kv ? VS : KS;
            constexpr int CT = kTtConv * 32;                     // threads of a tensor
            const int bF = kv ? (int)B_VF : (int)B_KF, bE = kv ? (int)B_VE : (int)B_KE;
            const auto* draft_rows = static_cast<const __nv_bfloat16*>(kv ? a.v_draft : a.k_draft);
            bool ok = true;
            int rst = 0, st = 0;                                 // stages of the rings, and the parities of their
            uint32_t rph = 0, ph = 1;                            // waits (a fresh ring's tiles are free)
            segments([&](int tile, int e0, int n, int, int, int) {
                const int bg = tile / g.tiles_bg, b = bg / g.Hkv;
                int len, nodes;
                tree_live(a.kv_len, a.n_nodes, g, b, &len, &nodes);
                ListWindow win;
                win.start(w.list + (size_t)tile * g.lcap, e0, e0 + n);
                for (int s = 0; s < n; ++s) {
                    win.to(e0 + s);
                    const int j = win.at(e0 + s);
                    const bool draft = j == kTreeDraft;
                    const int lim = draft ? nodes : j == kTreeOpen ? len % kBlock : kBlock;   // rows that are there
                    if (!draft) {
                        ok = ok && mbar_wait(bar(B_RF + rst), rph, abort_flag);
                    }
                    ok = ok && mbar_wait(bar(bE + st), ph, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) continue;
                    const uint8_t* rp = base_ptr + L::off_raw + rst * L::kRaw;
                    uint8_t* dst = base_ptr + (kv ? L::off_v : L::off_k) + st * L::kTile;
                    constexpr int IT = kBlock * CH / CT;
                    // chunks 2 c and 2 c + 1 of a row's half; the upper half's lanes store the odd chunk
                    // first, so the lanes of a phase fall in distinct banks
                    const int c = ct % CH, sw = c >> 2, c0 = (c & 3) * 2;
                    auto store = [&](int r, uint4 lo, uint4 hi) {
                        uint8_t* row = dst + sw * L::kHalf + r * 128;
                        *reinterpret_cast<uint4*>(row + (((c0 + sw) ^ (r & 7)) << 4)) = sw ? hi : lo;
                        *reinterpret_cast<uint4*>(row + (((c0 + 1 - sw) ^ (r & 7)) << 4)) = sw ? lo : hi;
                    };
                    auto convert = [&](uint4 x, uint32_t sb, uint4* lo, uint4* hi) {
                        const uint32_t f = sb == kScaleNaN ? 0x7fff7fffu : sb * 0x00800080u;   // 2^(s - 127), twice
                        e4m3x4_to_bf16x4(x.x, f, &lo->x, &lo->y);
                        e4m3x4_to_bf16x4(x.y, f, &lo->z, &lo->w);
                        e4m3x4_to_bf16x4(x.z, f, &hi->x, &hi->y);
                        e4m3x4_to_bf16x4(x.w, f, &hi->z, &hi->w);
                    };
                    const uint8_t* codes = rp + kv * L::kRawKV + ct * 16;
                    const uint8_t* scales = rp + 2 * L::kRawKV + kv * 64 + ct / CH;
                    constexpr int RS = CT / CH;                  // rows per round of the threads
                    if (j >= 0) {
                        constexpr int U4 = IT < 4 ? IT : 4;
#pragma unroll 1
                        for (int it0 = 0; it0 < IT; it0 += U4) {
                            uint4 x[U4];
                            uint32_t sb[U4];
#pragma unroll
                            for (int i = 0; i < U4; ++i) {
                                x[i] = *reinterpret_cast<const uint4*>(codes + (it0 + i) * CT * 16);
                                sb[i] = scales[(it0 + i) * RS];
                            }
#pragma unroll
                            for (int i = 0; i < U4; ++i) {
                                uint4 lo, hi;
                                convert(x[i], sb[i], &lo, &hi);
                                store((it0 + i) * RS + ct / CH, lo, hi);
                            }
                        }
                    } else {
                        // the open block's rows, or the draft's; zeros behind them
#pragma unroll 1
                        for (int it = 0; it < IT; ++it) {
                            const int r = it * RS + ct / CH;
                            uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                            if (r < lim) {
                                if (draft) {
                                    const uint4* p = reinterpret_cast<const uint4*>(draft_rows + ((size_t)bg * g.N + r) * D) + c * 2;
                                    lo = __ldg(p);
                                    hi = __ldg(p + 1);
                                } else {
                                    convert(*reinterpret_cast<const uint4*>(codes + it * CT * 16), scales[it * RS], &lo, &hi);
                                }
                            }
                            store(r, lo, hi);
                        }
                    }
                    fence_proxy_async_smem();
                    arrive(bar(bF + st));
                    if (!draft) {
                        arrive(bar(B_RE + rst));
                        if (++rst == kTtRaw) { rst = 0; rph ^= 1u; }
                    }
                    if (++st == NS) { st = 0; ph ^= 1u; }
                }
            });
        }
    } else {
        // ------------------------------------------------------------ softmax groups
        if constexpr (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 136;" ::: "memory");
        const int grp = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_col = grp * 64, o_col = L::colO + grp * D, p_col = L::colP + grp * 32;
        bool ok = true;
        auto wwait = [&](uint32_t bar_addr, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, abort_flag));
        };
        segments([&](int tile, int e0, int n, int gs0, int o0, int o1) {
            const int bg = tile / g.tiles_bg, b = bg / g.Hkv, row_g = (tile % g.tiles_bg) * kTreeRows + r;
            const bool in_tile = row_g < g.R;
            const size_t row = (size_t)bg * g.R + row_g;
            // everything that depends on the tile alone is on its way before any of it is used
            int len, nodes;
            tree_live(a.kv_len, a.n_nodes, g, b, &len, &nodes);
            auto entry = [&](int s) { return s < n ? __ldcg(w.list + (size_t)tile * g.lcap + e0 + s) : kTreeDraft; };
            const int s0 = (gs0 & 1) == grp ? 0 : 1;
            int j0 = entry(s0), j1 = entry(s0 + 2);
            const int node = in_tile ? row_g % g.N : 0;
            const size_t bn = (size_t)b * g.N;
            unsigned long long anc = in_tile ? __ldcg(w.anc + bn + node) : 0ull;
            const int dep = in_tile ? __ldcg(w.depth + bn + node) : 0;
            const float tau_m = in_tile ? __ldcg(w.tau + row) : 0.f;
            // group 0 brings the tile's rows of Q into TMEM, row r in lane r (zeros for rows it lacks)
            if (grp == 0) {
                const uint4* src = reinterpret_cast<const uint4*>(q + row * D);
                auto load = [&](int c) { return in_tile ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u); };
#pragma unroll
                for (int f = 0; f < D / 32; ++f) {
                    uint4 v[4];
                    uint32_t w16[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = load(f * 4 + c);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        w16[4 * c] = v[c].x; w16[4 * c + 1] = v[c].y;
                        w16[4 * c + 2] = v[c].z; w16[4 * c + 3] = v[c].w;
                    }
                    tmem_st16(lane_addr + L::colQ + f * 16, w16);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(bar(B_Q));
            }
            const int F = len / kBlock, rem = len % kBlock;
            if (node >= nodes) anc = 0ull;
            const bool valid = anc != 0ull;
            const bool warp_live = __any_sync(0xffffffffu, valid);
            const float tau_r = valid ? tau_m : __int_as_float(0x7fc00000);
            const float* xr = w.xs + row * g.cap;
            const bool crossed = valid && rem + dep >= kBlock;
            auto xval = [&](int j) { return valid && j >= 0 ? __ldcg(xr + j) : 0.f; };
            const float xF = crossed ? __ldcg(xr + F) : 0.f;
            float x0 = xval(j0);
            // log2 prior of the open block's keys: 1 while it is the own block
            const float lpo = !crossed ? 0.f : xF > tau_r ? e_pow * __log2f(xF - tau_r) : xF == xF ? -INFINITY : xF;
            float m_run = -INFINITY, l_run = 0.f;
            for (int s = s0; s < n; s += 2) {
                const int gs = gs0 + s, i2 = gs >> 1;
                const float x1 = xval(j1);                       // the next steps' values, on their way early
                const int j2 = entry(s + 4);
                const int j = j0;
                const float x = x0;
                j0 = j1; j1 = j2; x0 = x1;
                if (!(ok && wwait(bar(B_SF + grp), i2 & 1))) { ok = false; continue; }
                if (!warp_live) {
                    // no row of this warp is used; its lanes of S, P and O hold whatever they hold.  It
                    // still waits for the product before, so as not to count towards an earlier P
                    arrive(bar(B_SE + grp));
                    if (i2 >= 1 && !wwait(bar(B_PD + grp), (i2 - 1) & 1)) { ok = false; continue; }
                    arrive(bar(B_PF + grp));
                    continue;
                }
                float scale = sm2;
                tc_fence_after();
                float lp2;
                unsigned long long on = 0ull, low = 0ull;        // special entries: attended keys, those with prior lpo
                if (j >= 0) {
                    lp2 = valid && x > tau_r ? e_pow * __log2f(x - tau_r) : -INFINITY;
                } else {
                    // the open block's keys (those before the sequence's end), or the draft's (ancestors
                    // and self; those in a completed open block carry its prior)
                    if (j == kTreeOpen) {
                        on = low = (1ull << rem) - 1ull;
                    } else {
                        on = anc;
                        if (crossed)
                            for (int i = 0; i < nodes; ++i)
                                if (rem + w.depth[bn + i] < kBlock) low |= 1ull << i;
                    }
                    lp2 = valid ? 0.f : -INFINITY;
                }
                uint32_t sr[64];
                float mx = -INFINITY;
                // rows that do not attend this entry skip its scores: whole warps of them often do
                if (__any_sync(0xffffffffu, lp2 > -INFINITY)) {
                    if (j < 0) {
                        // finished logits in place of the scores, -inf where a key is not attended; back
                        // to TMEM 16 at a time, in a loop: rare code that is kept small
#pragma unroll 1
                        for (int c = 0; c < 64; c += 16) {
                            uint32_t t[16];
                            tmem_ld16(lane_addr + s_col + c, t);
                            tmem_wait_ld();
                            const uint32_t om = (uint32_t)(on >> c), lm = (uint32_t)(low >> c);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float v = __uint_as_float(t[i]) * sm2;
                                if ((lm >> i) & 1u) v = lpo == -INFINITY ? -INFINITY : v + lpo;
                                t[i] = __float_as_uint((om >> i) & 1u ? v : -INFINITY);
                            }
                            tmem_st16(lane_addr + s_col + c, t);
                        }
                        tmem_wait_st();
                        scale = 1.f;
                    }
                    tmem_ld<64>(lane_addr + s_col, sr);
                    tmem_wait_ld();
                    float m4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) m4[i] = fmaxf(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1]));
#pragma unroll
                    for (int i = 4; i < 32; ++i) m4[i & 3] = max3(m4[i & 3], __uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1]));
                    if (lp2 > -INFINITY) mx = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), scale, lp2);
                }
                tc_fence_before();
                arrive(bar(B_SE + grp));
                // Maxima leave NaN out, so an entry is not passed over by its maximum: a row may attend one key
                // of it alone (a root its own), and where that is no number the sum has to be NaN
                const bool active = lp2 > -INFINITY;
                float factor = 1.f;
                bool resc = false;
                if (mx > -INFINITY) {
                    if (m_run == -INFINITY) m_run = mx;
                    else if (mx > m_run + kTtLazy) { factor = exp2f(m_run - mx); m_run = mx; resc = true; }
                }
                const float c0 = m_run == -INFINITY ? lp2 : lp2 - m_run;
                const uint64_t sc2 = f2_pack(__float_as_uint(scale), __float_as_uint(scale));
                const uint64_t c2 = f2_pack(__float_as_uint(c0), __float_as_uint(c0));
                uint32_t pk[32];
                uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    pk[i] = 0u;
                    if (active) {
                        float v0, v1;
                        f2_unpack(f2_fma(f2_pack(sr[2 * i], sr[2 * i + 1]), sc2, c2), v0, v1);
                        v0 = fast_exp2(v0);
                        v1 = fast_exp2(v1);
                        sum2[i & 1] = f2_add(sum2[i & 1], f2_pack(__float_as_uint(v0), __float_as_uint(v1)));
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(v0, v1);
                        pk[i] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                }
                {
                    float a0, a1;
                    f2_unpack(f2_add(sum2[0], sum2[1]), a0, a1);
                    l_run = fmaf(l_run, factor, a0 + a1);
                }
                // the group's previous product has read P and written O
                if (i2 >= 1) {
                    if (!wwait(bar(B_PD + grp), (i2 - 1) & 1)) { ok = false; continue; }
                    tc_fence_after();
                }
                tmem_st32(lane_addr + p_col, pk);
                if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 2
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(lane_addr + o_col + c * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
                        tmem_st16(lane_addr + o_col + c * 16, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(bar(B_PF + grp));
            }
            if (tid == 0 && e0 == 0) w.offs[tile] = o0;          // for the merge of a split tile
            if (l_run != l_run && m_run == -INFINITY) m_run = 0.f;   // no score but NaN: the merge takes the sum up
            // ---- the two groups' states: (max, sum, output) of every row
            m_sh[grp][r] = m_run;
            l_sh[grp][r] = l_run;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const int gl = gs0 + n - 1;                          // last step; the other group's last is before it
            const bool both = n >= 2;
            bool done = ok;
            done = done && wwait(bar(B_PD + (gl & 1)), (gl >> 1) & 1);
            if (both) done = done && wwait(bar(B_PD + ((gl - 1) & 1)), ((gl - 1) >> 1) & 1);
            if (done && warp_live) {
                tc_fence_after();
                const bool has0 = both || (gl & 1) == 0, has1 = both || (gl & 1) == 1;
                const float m0 = has0 ? m_sh[0][r] : -INFINITY, m1 = has1 ? m_sh[1][r] : -INFINITY;
                const float M = fmaxf(m0, m1);
                const float w0 = m0 == -INFINITY ? 0.f : exp2f(m0 - M), w1 = m1 == -INFINITY ? 0.f : exp2f(m1 - M);
                const float l0 = l_sh[0][r], l1 = l_sh[1][r];
                // a sum that is NaN counts whatever its weight is
                const float den = (m0 == -INFINITY ? 0.f : l0 * w0) + (m1 == -INFINITY ? 0.f : l1 * w1);
                // whether the tile lies in this CTA's range
                const bool direct = sh.lo <= o0 && o1 <= sh.hi;
                // partial of a tile: (max, sum) per row, then the outputs as [dims / 4][row][4], which
                // the lanes of a warp (rows) write side by side
                float* pr = w.part + ((size_t)cta + tile) * kTreeRows * (D + 4);
                if (!direct && valid && grp == 0) *reinterpret_cast<float2*>(pr + 2 * r) = make_float2(M, den);
                const float inv = direct ? 1.0f / den : 1.0f;
                auto* out = static_cast<__nv_bfloat16*>(a.out) + row * D;
#pragma unroll 2
                for (int c = 0; c < D / 32; ++c) {
                    const int col = grp * (D / 2) + c * 16;      // the groups share the row's columns
                    uint32_t p0[16], p1[16];
                    tmem_ld16(lane_addr + L::colO + col, p0);
                    tmem_ld16(lane_addr + L::colO + D + col, p1);
                    tmem_wait_ld();
                    if (valid) {
                        float f[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float v = w0 > 0.f ? __uint_as_float(p0[i]) * w0 : 0.f;
                            if (w1 > 0.f) v = fmaf(__uint_as_float(p1[i]), w1, v);
                            f[i] = v * inv;
                        }
                        if (direct) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t pk[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(f[8 * i + 2 * k], f[8 * i + 2 * k + 1]);
                                    pk[k] = *reinterpret_cast<const uint32_t*>(&h2);
                                }
                                *reinterpret_cast<uint4*>(out + col + 8 * i) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<float4*>(pr + 4 * kTreeRows + ((col / 4 + i) * kTreeRows + r) * 4) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                        }
                    }
                }
            }
            // Q, O and the maxima are free for the next segment
            tc_fence_before();
            asm volatile("bar.sync 1, 256;" ::: "memory");
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && abort_sh) atomicOr(&w.hdr->status, kStWaitTimeout);
}

// Merges the partials of a tile that several CTAs share.  A CTA takes 1024 / (D PG) rows: a warp
// makes the weights of a row's pieces (lanes over the pieces), a thread sums four dims of a row over
// every PG-th piece, eight of them in flight, and the PG sums are added in order.  The lanes of a
// warp read side by side in the partials' [dims / 4][row] order.  Which pieces there are follows from the
// lists' lengths, which are there before the attention ends.
template <int D, int PG>
__global__ void __launch_bounds__(256)
tree_combine_kernel(TreeArgs a, TreeWork w, TreeGeom g, int nctas) {
    constexpr int RPC = 1024 / (D * PG), RW = (RPC + 7) / 8, KB = 8;   // RW: rows whose weights a warp makes
    __shared__ float wt_sh[RPC][kDecodeMaxCtas], inv_sh[RPC];
    __shared__ float4 sum_sh[PG][256 / PG];
    __shared__ int place_sh[16];
    const int per_tile = (min(g.R, kTreeRows) + RPC - 1) / RPC;
    const int tile = blockIdx.x / per_tile, r0 = (blockIdx.x % per_tile) * RPC;
    const int bg = tile / g.tiles_bg, b = bg / g.Hkv, row0 = (tile % g.tiles_bg) * kTreeRows + r0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ListPlace at = list_place<256>(w.count, w.offs, g.tiles, tile, place_sh);
    const ListSplit sp(at.U, g.tiles, nctas, 0);
    int c0 = 0, np = 1;
    if (at.n > 0) {
        c0 = sp.cta_of(at.o0);
        np = sp.cta_of(at.o0 + at.n - 1) - c0 + 1;
    }
    int len, nodes;
    const bool live = tree_live(a.kv_len, a.n_nodes, g, b, &len, &nodes);
    bool there[RW];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
        const int row = row0 + warp + 8 * k, node = row % g.N;
        there[k] = warp + 8 * k < RPC && row < g.R && node < nodes && __ldcg(w.anc + (size_t)b * g.N + node) != 0ull;
    }
    pdl_wait();
    if (np == 1 || !live || row0 >= g.R) return;                 // finished by one CTA, or nothing to do
    const float* p = w.part + ((size_t)c0 + tile) * kTreeRows * (D + 4);
    const size_t step = (size_t)kTreeRows * (D + 4);
    const int rr = tid % RPC, c4 = tid / RPC % (D / 4), pg = tid / (256 / PG);
    const float* po = p + 4 * kTreeRows + ((size_t)c4 * kTreeRows + r0 + rr) * 4;
    float4 v[KB];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < KB; ++k)
            if (i0 + k * PG < np) v[k] = __ldcg(reinterpret_cast<const float4*>(po + (i0 + k * PG) * step));
    };
    load(pg);
#pragma unroll
    for (int k = 0; k < RW; ++k) {
        const int rw = warp + 8 * k;
        if (rw >= RPC) break;
        float den = -1.f;                                        // no such row, or none to merge
        if (there[k]) {
            const float* ph = p + 2 * (r0 + rw);
            auto stats = [&](int i) { return i < np ? __ldcg(reinterpret_cast<const float2*>(ph + i * step)) : make_float2(-INFINITY, 0.f); };
            const float2 first = stats(lane);
            float M = first.x;
            for (int i = lane + 32; i < np; i += 32) M = fmaxf(M, stats(i).x);
            M = warp_max(M);
            den = 0.f;
            for (int i = lane; i < np; i += 32) {
                const float2 ml = i < 32 ? first : stats(i);
                const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
                wt_sh[rw][i] = wt;
                den = fmaf(ml.y, wt, den);
            }
            den = warp_sum(den);
        }
        if (lane == 0) inv_sh[rw] = den < 0.f ? -1.f : 1.0f / den;
    }
    __syncthreads();
    const float inv = inv_sh[rr];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!(inv < 0.f)) {
        for (int i0 = pg;;) {
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                const int i = i0 + k * PG;
                if (i < np) {
                    const float wt = wt_sh[rr][i];
                    acc.x = fmaf(v[k].x, wt, acc.x);
                    acc.y = fmaf(v[k].y, wt, acc.y);
                    acc.z = fmaf(v[k].z, wt, acc.z);
                    acc.w = fmaf(v[k].w, wt, acc.w);
                }
            }
            i0 += KB * PG;
            if (i0 >= np) break;
            load(i0);
        }
    }
    if constexpr (PG > 1) {
        sum_sh[pg][tid % (256 / PG)] = acc;
        __syncthreads();
        if (pg > 0) return;
#pragma unroll
        for (int k = 1; k < PG; ++k) {
            const float4 o = sum_sh[k][tid];
            acc.x += o.x; acc.y += o.y; acc.z += o.z; acc.w += o.w;
        }
    }
    if (inv < 0.f) return;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + ((size_t)bg * g.R + row0 + rr) * D + c4 * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <int D, bool Q8>
static cudaError_t launch_t(const TreeArgs& a, const TreeWork& w, const TreeGeom& g, float e_pow, float sm2, int nctas,
                            cudaStream_t stream) {
    CUtensorMap tk = {}, tv = {}, tkd = {}, tvd = {};
    if constexpr (!Q8) {
        const unsigned long long rows = (unsigned long long)g.B * g.Hkv * g.Tmax, drows = (unsigned long long)g.B * g.Hkv * g.N;
        if (!make_tmap_bf16(&tk, a.k_cache, rows, D, kBlock) || !make_tmap_bf16(&tv, a.v_cache, rows, D, kBlock) ||
            !make_tmap_bf16(&tkd, a.k_draft, drows, D, kBlock) || !make_tmap_bf16(&tvd, a.v_draft, drows, D, kBlock))
            return cudaErrorInvalidValue;
    }
    const int sm = (int)TtLayout<D, Q8>::bytes;
    cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    if (e != cudaSuccess) return e;
    const PdlConfig ca(nctas, kTtThreads<Q8>, sm, stream);
    e = cudaLaunchKernelEx(&ca.cfg, tree_attn_kernel<D, Q8>, tk, tv, tkd, tvd, a, w, g, e_pow, sm2);
    if (e != cudaSuccess) return e;
    // few tiles: long lists of pieces and few CTAs, so four threads share a sum (one of 128 rows and 37
    // pieces a row: 14 us without); many tiles have a few pieces each
    const int rows = g.R < kTreeRows ? g.R : kTreeRows;
    const bool wide = (long long)g.tiles * rows * D / 1024 <= nctas;
    const int rpc = 1024 / D / (wide ? 4 : 1);
    const PdlConfig cc((unsigned)g.tiles * ((rows + rpc - 1) / rpc), 256, 0, stream);
    e = wide ? cudaLaunchKernelEx(&cc.cfg, tree_combine_kernel<D, 4>, a, w, g, nctas)
             : cudaLaunchKernelEx(&cc.cfg, tree_combine_kernel<D, 1>, a, w, g, nctas);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_attn(const TreeArgs& a, const TreeWork& w, const TreeGeom& g, float e_pow, float sm2, int nctas,
                             cudaStream_t stream) {
    if (nctas < 1 || nctas > kDecodeMaxCtas) return cudaErrorInvalidValue;
    if (g.d == 128) return a.k_scale ? launch_t<128, true>(a, w, g, e_pow, sm2, nctas, stream)
                                     : launch_t<128, false>(a, w, g, e_pow, sm2, nctas, stream);
    return a.k_scale ? launch_t<64, true>(a, w, g, e_pow, sm2, nctas, stream)
                     : launch_t<64, false>(a, w, g, e_pow, sm2, nctas, stream);
}

}  // namespace dash
