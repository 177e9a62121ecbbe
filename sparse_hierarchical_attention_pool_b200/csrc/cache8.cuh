// cache8.cuh -- the 8-bit KV cache: format and conversions.
//
// A cached row (the d keys or values of one token and KV head) is d e4m3 codes and one scale
// byte s; element i stands for code_i 2^(s - 127).  For a row x with largest finite magnitude
// amax, the exponent is the least e >= kScaleMin with amax <= 448 2^e (448 is the largest e4m3
// number, so nothing saturates), code_i = e4m3(x_i 2^-e) rounded to nearest even, s = e + 127.
// Scales are powers of two: the product x_i 2^-e is exact, so each element is rounded once, to
// e4m3's 4 significant bits (relative 2^-4 down to 2^-6 2^e, absolute 2^-10 2^e below), and
// every held value is exact in bf16 (4 significant bits, and kScaleMin keeps the smallest,
// 2^-9 2^-118 = 2^-127, on bf16's subnormal grid of 2^-133; at e = 120, the largest, magnitudes saturate at 240 2^120).  One scale per row suffices: e4m3
// is a floating-point format whose 17 binades cover a row's spread; finer scales would gain
// only elements more than 2^14 below the row's largest.
// A row with a NaN or an infinity gets s = kScaleNaN and stands for NaN in every element (its
// non-finite elements' codes are 0): codes are never NaN, so a product with weight zero is zero.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dash {

constexpr int kScaleMin = -118;
constexpr unsigned kHeldTop = 0x7f70u;          // bf16 bits of the largest held magnitude, 240 2^120 (256 2^120 would be no bf16 number)
constexpr unsigned kScaleNaN = 255u;

// 2^(s - 127) for the scale bytes the cache holds (9 .. 247), NaN for kScaleNaN
__device__ __forceinline__ float scale_value(unsigned s) {
    return __uint_as_float(s == kScaleNaN ? 0x7fc00000u : s << 23);
}

// exponent e of a row whose largest finite magnitude is amax (0 included)
__device__ __forceinline__ int scale_exponent(float amax) {
    const unsigned u = __float_as_uint(amax);
    const int k = (int)(u >> 23) - 127;                       // amax = 1.m 2^k; 448 = 1.75 2^8
    const int e = (u & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7;
    return max(e, kScaleMin);
}

// two codes (low byte first) as an f16 pair: every e4m3 number is exact in f16
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}

// four codes times f, as fp32
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float f, float* o) {
    const uint32_t lo = e4m3x2_to_f16x2((uint16_t)w), hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    o[0] = a.x * f; o[1] = a.y * f; o[2] = b.x * f; o[3] = b.y * f;
}

}  // namespace dash
