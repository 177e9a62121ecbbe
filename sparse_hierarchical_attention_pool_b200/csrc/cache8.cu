// cache8.cu -- writing rows to the 8-bit KV cache, keeping its block summaries, and reading it
// back (format: cache8.cuh).
#include "cache8.cuh"
#include "kernels.h"

namespace dash {

// ------------------------------------------------------------------ append
//
// One CTA of 8 warps per (b, KV head, 64-key block that the call touches): warp w holds the
// block's rows 8 w .. 8 w + 7, D / 8 lanes per row with 8 elements each, all loads issued
// before the first use.  A row's largest magnitude is a butterfly over its lanes.  Rows of the
// block that were in the cache before (only the first block of a sequence has any) are read
// back when the call completes the block, so the summary is the mean of the values that the
// cache holds, whatever calls wrote them: it depends on the cache alone and stays right when
// rows are written again (a drafted path that was not accepted).
template <int D>
__global__ void __launch_bounds__(256)
cache_append_kernel(const __nv_bfloat16* __restrict__ k_new, const __nv_bfloat16* __restrict__ v_new,
                    const int* __restrict__ src, const int* __restrict__ n_new, const int* __restrict__ kv_len,
                    uint8_t* __restrict__ kc, uint8_t* __restrict__ vc, uint8_t* __restrict__ ks,
                    uint8_t* __restrict__ vs, float* __restrict__ ksum, int Hkv, int n_rows, int n, int Tmax) {
    constexpr int LPR = D / 8;                 // lanes per row
    constexpr int RPS = 32 / LPR;              // rows per warp-wide load
    constexpr int STEPS = 8 / RPS;             // loads per warp and tensor
    __shared__ float red[8][D];
    const int bg = blockIdx.x, b = bg / Hkv;
    const int L = kv_len[b], m = n_new ? n_new[b] : n;
    if (L < 0 || m < 0 || m > n || L > Tmax - m) return;             // not a valid append: nothing written
    const int j = L / kBlock + (int)blockIdx.y;
    const int t0 = max(L, j * kBlock), t1 = min(L + m, j * kBlock + kBlock);
    if (t0 >= t1) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int* sb = src ? src + (size_t)b * n : nullptr;
    if (sb) {
        // a row index outside k_new refuses the sequence
        int bad = 0;
        for (int i = tid; i < m; i += 256) bad |= (unsigned)sb[i] >= (unsigned)n_rows;
        if (__syncthreads_or(bad)) return;
    }
    const bool want = ksum && j * kBlock + kBlock <= L + m;          // the call completes this block
    const int cg = lane % LPR;
    const size_t row0 = (size_t)bg * Tmax;
    uint4 kx[STEPS], vx[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int t = j * kBlock + warp * 8 + s * RPS + lane / LPR;
        kx[s] = vx[s] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= t0 && t < t1) {
            const size_t r = (size_t)bg * n_rows + (sb ? sb[t - L] : t - L);
            kx[s] = __ldg(reinterpret_cast<const uint4*>(k_new + r * D) + cg);
            vx[s] = __ldg(reinterpret_cast<const uint4*>(v_new + r * D) + cg);
        } else if (want && t < t0) {
            const uint2 c = *reinterpret_cast<const uint2*>(kc + (row0 + t) * D + cg * 8);
            kx[s].x = c.x; kx[s].y = c.y;
            vx[s].x = ks[row0 + t];
        }
    }
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    // quantises one row (all lanes of the warp take part); f: the scale as a number
    auto quantise = [&](const uint4& x, uint2* code, unsigned* scale) {
        float f[8], amax = 0.f;
        bf16x8_to_float(x, f);
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool fin = fabsf(f[i]) < INFINITY;
            bad |= !fin;
            f[i] = fin ? f[i] : 0.f;
            amax = fmaxf(amax, fabsf(f[i]));
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const unsigned votes = __ballot_sync(0xffffffffu, bad) >> (lane / LPR * LPR);
        bad = LPR == 32 ? votes != 0u : (votes & ((1u << LPR) - 1u)) != 0u;
        const int e = scale_exponent(amax);
        const float inv = __uint_as_float((unsigned)(127 - e) << 23);
        if (e == kScaleMax) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -kHeldMax), kHeldMax);
        }
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        *code = make_uint2(w[0], w[1]);
        *scale = bad ? kScaleNaN : (unsigned)(e + 127);
    };
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int t = j * kBlock + warp * 8 + s * RPS + lane / LPR;
        const bool fresh = t >= t0 && t < t1;
        uint2 ck, cv;
        unsigned sk, sv;
        quantise(kx[s], &ck, &sk);
        quantise(vx[s], &cv, &sv);
        if (fresh) {
            *reinterpret_cast<uint2*>(kc + (row0 + t) * D + cg * 8) = ck;
            *reinterpret_cast<uint2*>(vc + (row0 + t) * D + cg * 8) = cv;
            if (cg == 0) { ks[row0 + t] = (uint8_t)sk; vs[row0 + t] = (uint8_t)sv; }
        } else {
            ck = make_uint2(kx[s].x, kx[s].y);
            sk = vx[s].x;
        }
        if (want) {
            float f[8];
            const float sc = scale_value(sk);
            e4m3x4_to_float(ck.x, sc, f);
            e4m3x4_to_float(ck.y, sc, f + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
    }
    if (!want) return;                                               // uniform over the CTA
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane < LPR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) red[warp][cg * 8 + i] = acc[i];
    }
    __syncthreads();
    if (tid < D) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += red[w][tid];
        ksum[((size_t)bg * (Tmax / kBlock) + j) * D + tid] = sum * (1.0f / kBlock);
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
// Thread = 16 codes of one row (one 16-byte load, two 16-byte stores) of K and of V, for
// kReadIter rows.  The product code * 2^(s - 127) is exact in fp32 and in bf16.
constexpr int kReadIter = 2;

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
    const int i0 = (int)blockIdx.y * RPI * kReadIter + threadIdx.x / LPR;
    const size_t row0 = (size_t)bg * Tmax;
    uint4 c[kReadIter][2];
    unsigned s[kReadIter][2];
#pragma unroll
    for (int it = 0; it < kReadIter; ++it) {
        const int i = i0 + it * RPI;
        const long long t = (long long)first + i;
        c[it][0] = c[it][1] = make_uint4(0u, 0u, 0u, 0u);
        s[it][0] = s[it][1] = 127u;
        if (i < n && t >= 0 && t < end) {
            c[it][0] = __ldg(reinterpret_cast<const uint4*>(kc + (row0 + t) * D) + cg);
            c[it][1] = __ldg(reinterpret_cast<const uint4*>(vc + (row0 + t) * D) + cg);
            s[it][0] = __ldg(ks + row0 + t);
            s[it][1] = __ldg(vs + row0 + t);
        }
    }
#pragma unroll
    for (int it = 0; it < kReadIter; ++it) {
        const int i = i0 + it * RPI;
        if (i >= n) break;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const float f = scale_value(s[it][kv]);
            const uint32_t w[4] = {c[it][kv].x, c[it][kv].y, c[it][kv].z, c[it][kv].w};
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
}

cudaError_t launch_cache_read(const void* kc, const void* vc, const void* ks, const void* vs, const int* start,
                              const int* kv_len, void* ko, void* vo, int B, int Hkv, int n, int Tmax, int d,
                              cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    const int rows = 256 / (d / 16) * kReadIter;
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
