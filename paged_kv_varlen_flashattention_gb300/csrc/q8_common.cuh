// The 8-bit cache format: e4m3 codes with one f32 scale for each page and kv head of K and of V;
// an element's value is code x scale.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"

namespace pa {

constexpr float kE4m3Max = 448.f;
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

// The least power of two, 2^-100 at least, with which a finite absmax is at most 448 = 1.75 x 2^8:
// from the bits of absmax = 1.m x 2^E, E - 8 if 1.m <= 1.75 and E - 7 otherwise.
__device__ __forceinline__ float pow2_scale(float absmax) {
    const int bits = __float_as_int(absmax);
    int k = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    k = max(k, kScaleExpMin);
    return __int_as_float((k + 127) << 23);
}

}  // namespace pa
