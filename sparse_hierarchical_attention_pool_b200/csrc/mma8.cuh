// mma8.cuh -- what a step over the 8-bit KV cache adds to mma_sync.cuh and sm100.cuh: products of e4m3 and f16
// operands, and tensor maps of bytes.
#pragma once

#include "mma_sync.cuh"
#include "sm100.cuh"

namespace dash {

// make_tmap_bf16's counterpart over a row-major [rows, d] matrix of bytes (d = 64 or 128): boxes of whole rows,
// swizzled over a row's width (d = 128: 128-byte, d = 64: 64-byte swizzle).
bool make_tmap_u8(CUtensorMap* m, const void* ptr, unsigned long long rows, int d, int box_rows);

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8x8 matrix of 16-bit elements held as an mma fragment, transposed
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

}  // namespace dash
