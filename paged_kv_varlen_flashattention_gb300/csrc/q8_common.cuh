// The 8-bit cache format: e4m3 codes with one f32 scale for each page and kv head of K and of V;
// an element's value is code x scale.
#pragma once

#include <atomic>
#include <cuda_fp16.h>

#include "device_common.cuh"

namespace pa {

// Dynamic shared memory of a kernel, set once for each device that launches it.
template <typename K>
cudaError_t set_shared_memory(K kernel, int bytes, std::atomic<uint64_t>& devices) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (devices.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

constexpr int kScaleExpMin = -100;  // the smallest scale an append gives a page, and a read sees, is 2^-100

// Two fp32 values rounded to e4m3 (to nearest even, beyond 448 to 448): `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (low 16 bits of w) as two halves: exact, every e4m3 value is an f16 value.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
// The same for the high 16 bits of w.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_half2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Remainder terms: two fp32 values as e4m3 codes, and what the codes leave of them.
__device__ __forceinline__ uint32_t e4m3x2_take(float& lo, float& hi) {
    const uint32_t c = e4m3x2(lo, hi);
    const uint32_t h = e4m3x2_to_half2(c);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    lo -= f.x;
    hi -= f.y;
    return c;
}

// c (+)= A B of e4m3 fragments: A 16 x 32 (row-major), B 32 x 8 (column-major), fp32 accumulation.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two 16 x 16 byte matrices transposed: lane i gives the address of row i of the first (i < 16) or row
// i - 16 of the second; of each, lane 4 n + t gets rows 4 t .. 4 t + 3 of column n (r0, r2) and of
// column n + 8 (r1, r3): the B fragment of mma_e4m3 with the rows as k.
__device__ __forceinline__ void ldsm_b8_x2_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// The least power of two, 2^-100 at least, with which a finite absmax is at most 448 = 1.75 x 2^8:
// from the bits of absmax = 1.m x 2^E, E - 8 if 1.m <= 1.75 and E - 7 otherwise.
__device__ __forceinline__ float pow2_scale(float absmax) {
    const int bits = __float_as_int(absmax);
    int k = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    k = max(k, kScaleExpMin);
    return __int_as_float((k + 127) << 23);
}

}  // namespace pa
