// cache8.cu -- writing rows to the 8-bit KV cache, keeping its block summaries, and reading it
// back (format: cache8.cuh).
#include "cache8.cuh"
#include "kernels.h"

namespace dash {

// ------------------------------------------------------------------ append
//
// One CTA of 8 warps per (b, KV head, 64-key block that the call touches): warp w holds the
// block's rows 8 w .. 8 w + 7, D / 16 lanes per row with two chunks of 8 elements each, all loads
// issued before the first use.  A row's largest magnitude is a butterfly over its lanes.  Rows of the
// block that were in the cache before (only the first block of a sequence has any) are read
// back when the call completes the block, so the summary is the mean of the values that the
// cache holds, whatever calls wrote them: it depends on the cache alone and stays right when
// rows are written again (a drafted path that was not accepted).
// 4,096 rows of 4 x 8 heads of 128 dims (101 MB) take 23.5 us, 4.3 TB/s.  Neither instructions nor bytes fill
// it (60 % of the issue slots, 40 % of the DRAM's, most stalls on the loads: a CTA loads, works and stores once,
// in 2.8 waves); with 8 elements a lane, whose butterflies and exponents weigh twice as much, and comparisons
// element by element it took 30.6 us.
template <int D>
__global__ void __launch_bounds__(256)
cache_append_kernel(const __nv_bfloat16* __restrict__ k_new, const __nv_bfloat16* __restrict__ v_new,
                    const int* __restrict__ src, const int* __restrict__ n_new, const int* __restrict__ kv_len,
                    uint8_t* __restrict__ kc, uint8_t* __restrict__ vc, uint8_t* __restrict__ ks,
                    uint8_t* __restrict__ vs, float* __restrict__ ksum, int Hkv, int n_rows, int n, int Tmax) {
    constexpr int LPR = D / 16;                // lanes per row
    constexpr int RPS = 32 / LPR;              // rows per warp-wide load
    constexpr int STEPS = 8 / RPS;             // steps per warp and tensor
    __shared__ float red[8 * RPS][D];
    const int bg = blockIdx.x, b = bg / Hkv;
    const int L = kv_len[b], m = n_new ? n_new[b] : n;
    if (L < 0 || m < 0 || m > n || L > Tmax - m) return;             // not a valid append: nothing written
    const int j = L / kBlock + (int)blockIdx.y;
    const int t0 = max(L, j * kBlock), t1 = min(L + m, j * kBlock + kBlock);
    if (t0 >= t1) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int* sb = src ? src + (size_t)b * n : nullptr;
    if (sb) {
        // a row index outside k_new refuses the sequence; every CTA looks at the whole list (a path has up to 64 entries)
        int bad = 0;
        for (int i = tid; i < m; i += 256) bad |= (unsigned)sb[i] >= (unsigned)n_rows;
        if (__syncthreads_or(bad)) return;
    }
    const bool want = ksum && j * kBlock + kBlock <= L + m;          // the call completes this block
    const int cg = lane % LPR, rl = lane / LPR;
    const size_t row0 = (size_t)bg * Tmax;
    // chunk h of a lane: elements 8 (cg + h LPR) .. + 7 of its row
    uint4 kx[STEPS][2], vx[STEPS][2];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int t = j * kBlock + warp * 8 + s * RPS + rl;
#pragma unroll
        for (int h = 0; h < 2; ++h) kx[s][h] = vx[s][h] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= t0 && t < t1) {
            const size_t r = (size_t)bg * n_rows + (sb ? sb[t - L] : t - L);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                kx[s][h] = __ldg(reinterpret_cast<const uint4*>(k_new + r * D) + cg + h * LPR);
                vx[s][h] = __ldg(reinterpret_cast<const uint4*>(v_new + r * D) + cg + h * LPR);
            }
        } else if (want && t < t0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 c = *reinterpret_cast<const uint2*>(kc + (row0 + t) * D + (cg + h * LPR) * 8);
                kx[s][h].x = c.x; kx[s][h].y = c.y;
            }
            vx[s][0].x = ks[row0 + t];
        }
    }
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    // Quantises one row (all lanes of the warp take part).  A bf16's bits without the sign order like
    // its magnitude, so the largest of a row is an integer maximum, two elements at once.
    auto quantise = [&](uint4 (&x)[2], uint2 (&code)[2], unsigned* scale) {
        constexpr unsigned kAbs = 0x7fff7fffu, kInf = 0x7f80u;
        auto largest = [&]() {
            unsigned m = 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[h].x & kAbs, x[h].y & kAbs), __vmaxu2(x[h].z & kAbs, x[h].w & kAbs)));
            m = max(m >> 16, m & 0xffffu);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            return m;
        };
        unsigned m = largest();
        const bool bad = m >= kInf;                                  // a NaN or an infinity in the row
        if (__any_sync(0xffffffffu, m > kHeldTop)) {
            // zeros for elements that are no numbers, and the largest magnitude that is held
            auto finite = [&](uint32_t w) {
                w &= ~__vcmpgeu2(w & kAbs, kInf * 0x10001u);
                return (w & ~kAbs) | __vminu2(w & kAbs, kHeldTop * 0x10001u);
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) x[h] = make_uint4(finite(x[h].x), finite(x[h].y), finite(x[h].z), finite(x[h].w));
            m = largest();
        }
        const int e = scale_exponent(__uint_as_float(m << 16));
        const float inv = __uint_as_float((unsigned)(127 - e) << 23);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[8];
            uint32_t w[2];
            bf16x8_to_float(x[h], f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                w[i] = lo | (hi << 16);
            }
            code[h] = make_uint2(w[0], w[1]);
        }
        *scale = bad ? kScaleNaN : (unsigned)(e + 127);
    };
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int t = j * kBlock + warp * 8 + s * RPS + rl;
        const bool fresh = t >= t0 && t < t1;
        uint2 ck[2], cv[2], old[2] = {make_uint2(kx[s][0].x, kx[s][0].y), make_uint2(kx[s][1].x, kx[s][1].y)};
        unsigned sk, sv;
        const unsigned old_scale = vx[s][0].x;
        quantise(kx[s], ck, &sk);
        quantise(vx[s], cv, &sv);
        if (fresh) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                *reinterpret_cast<uint2*>(kc + (row0 + t) * D + (cg + h * LPR) * 8) = ck[h];
                *reinterpret_cast<uint2*>(vc + (row0 + t) * D + (cg + h * LPR) * 8) = cv[h];
            }
            if (cg == 0) { ks[row0 + t] = (uint8_t)sk; vs[row0 + t] = (uint8_t)sv; }
        } else {
            ck[0] = old[0];
            ck[1] = old[1];
            sk = old_scale;
        }
        if (want) {
            // code * 2^(s - 127) is exact, so one fused operation adds what the cache holds; a 64th of it, which is
            // exact too (2^-133 at least), so that keys near the largest held number do not add up to infinity
            const float sc = scale_value(sk) * (1.0f / kBlock);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[8];
                e4m3x4_to_float(ck[h].x, 1.0f, f);
                e4m3x4_to_float(ck[h].y, 1.0f, f + 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[h * 8 + i] = fmaf(f[i], sc, acc[h * 8 + i]);
            }
        }
    }
    if (!want) return;                                               // uniform over the CTA
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<float4*>(&red[warp * RPS + rl][(cg + h * LPR) * 8 + i]) =
                make_float4(acc[h * 8 + i], acc[h * 8 + i + 1], acc[h * 8 + i + 2], acc[h * 8 + i + 3]);
    __syncthreads();
    if (tid < D) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8 * RPS; ++w) sum += red[w][tid];
        ksum[((size_t)bg * (Tmax / kBlock) + j) * D + tid] = sum;
    }
}

cudaError_t launch_cache_append(const void* k_new, const void* v_new, const int* src, const int* n_new,
                                const int* kv_len, void* kc, void* vc, void* ks, void* vs, float* ksum, int B,
                                int Hkv, int n_rows, int n, int Tmax, int d, cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    // a run of n rows that starts anywhere in a block touches at most this many blocks
    const dim3 grid((unsigned)(B * Hkv), (unsigned)((n + kBlock - 2) / kBlock + 1));
    const auto* kn = static_cast<const __nv_bfloat16*>(k_new);
    const auto* vn = static_cast<const __nv_bfloat16*>(v_new);
    auto* k8 = static_cast<uint8_t*>(kc);
    auto* v8 = static_cast<uint8_t*>(vc);
    auto* s8 = static_cast<uint8_t*>(ks);
    auto* t8 = static_cast<uint8_t*>(vs);
    if (d == 128) cache_append_kernel<128><<<grid, 256, 0, stream>>>(kn, vn, src, n_new, kv_len, k8, v8, s8, t8, ksum, Hkv, n_rows, n, Tmax);
    else cache_append_kernel<64><<<grid, 256, 0, stream>>>(kn, vn, src, n_new, kv_len, k8, v8, s8, t8, ksum, Hkv, n_rows, n, Tmax);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ read
//
// Thread = 16 codes of one row (one 16-byte load, two 16-byte stores) of K and of V.  The product
// code * 2^(s - 127) is exact in fp32 and in bf16.  Bound by HBM: 98,304 rows of 8 heads of 128
// dims (606 MB) take 108 us, 5.6 TB/s, 86 % of what a plain copy reaches; two rows a thread took
// 110 us and four 116.
template <int D>
__global__ void __launch_bounds__(256)
cache_read_kernel(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc, const uint8_t* __restrict__ ks,
                  const uint8_t* __restrict__ vs, const int* __restrict__ start, const int* __restrict__ kv_len,
                  __nv_bfloat16* __restrict__ ko, __nv_bfloat16* __restrict__ vo, int Hkv, int n, int Tmax) {
    constexpr int LPR = D / 16, RPI = 256 / LPR;
    const int bg = blockIdx.x, b = bg / Hkv;
    const int first = start ? start[b] : 0;
    const int end = kv_len ? min(kv_len[b], Tmax) : Tmax;
    const int cg = threadIdx.x % LPR;
    const int i = (int)blockIdx.y * RPI + threadIdx.x / LPR;
    if (i >= n) return;
    const long long t = (long long)first + i;
    const size_t row = (size_t)bg * Tmax + (size_t)t;                // used where t is a row of the sequence
    uint4 c[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    unsigned s[2] = {127u, 127u};
    if (t >= 0 && t < end) {
        c[0] = __ldg(reinterpret_cast<const uint4*>(kc + row * D) + cg);
        c[1] = __ldg(reinterpret_cast<const uint4*>(vc + row * D) + cg);
        s[0] = __ldg(ks + row);
        s[1] = __ldg(vs + row);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float f = scale_value(s[kv]);
        const uint32_t w[4] = {c[kv].x, c[kv].y, c[kv].z, c[kv].w};
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
            e4m3x4_to_float(w[q], f, v);
            const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), e = __floats2bfloat162_rn(v[2], v[3]);
            o[2 * q] = *reinterpret_cast<const uint32_t*>(&a);
            o[2 * q + 1] = *reinterpret_cast<const uint32_t*>(&e);
        }
        uint4* dst = reinterpret_cast<uint4*>((kv ? vo : ko) + ((size_t)bg * n + i) * D) + cg * 2;
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

cudaError_t launch_cache_read(const void* kc, const void* vc, const void* ks, const void* vs, const int* start,
                              const int* kv_len, void* ko, void* vo, int B, int Hkv, int n, int Tmax, int d,
                              cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    const int rows = 256 / (d / 16);
    const dim3 grid((unsigned)(B * Hkv), (unsigned)((n + rows - 1) / rows));
    const auto* k8 = static_cast<const uint8_t*>(kc);
    const auto* v8 = static_cast<const uint8_t*>(vc);
    const auto* s8 = static_cast<const uint8_t*>(ks);
    const auto* t8 = static_cast<const uint8_t*>(vs);
    auto* kb = static_cast<__nv_bfloat16*>(ko);
    auto* vb = static_cast<__nv_bfloat16*>(vo);
    if (d == 128) cache_read_kernel<128><<<grid, 256, 0, stream>>>(k8, v8, s8, t8, start, kv_len, kb, vb, Hkv, n, Tmax);
    else cache_read_kernel<64><<<grid, 256, 0, stream>>>(k8, v8, s8, t8, start, kv_len, kb, vb, Hkv, n, Tmax);
    return cudaGetLastError();
}

}  // namespace dash
