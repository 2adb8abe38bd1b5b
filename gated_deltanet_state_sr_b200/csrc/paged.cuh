// Shared by the kernels of the paged 8-bit key/value cache: e4m3 conversions
// and the scale of a block.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace sr {
namespace paged {

// The exponents a block's power-of-two scale may take.  They bound the ratio of
// two blocks' scales by 2^64, which fp32 holds beside any weight that counts.
constexpr int kScaleExpMin = -32, kScaleExpMax = 32;

// Least e with amax <= 449 * 2^e, clamped.  449, not 448 (the largest e4m3
// value): what lies between rounds to 448 anyway, and 449 * 2^e has nine
// significant bits, so no bf16 input sits on the border, where the last bit of
// an fp32 product would decide.  449 = 0.876953125 * 2^9.
__device__ __forceinline__ int scale_exp(float amax) {
    if (!(amax > 0.f)) return kScaleExpMin;
    int e;
    const float m = frexpf(amax, &e);
    e = m <= 0.876953125f ? e - 9 : e - 8;
    return min(max(e, kScaleExpMin), kScaleExpMax);
}

// Two floats to e4m3 (round to nearest even, clipped at +-448).  Infinities and
// NaN become the NaN byte: x + 0 x keeps every finite x.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(fmaf(a, 0.f, a), fmaf(b, 0.f, b)), __NV_SATFINITE,
                                             __NV_E4M3));
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    return to_e4m3x2(a, b) | (to_e4m3x2(c, d) << 16);
}
// The same without the care for infinities, which are clipped too.
__device__ __forceinline__ uint32_t clipped_e4m3x4(float a, float b, float c, float d) {
    return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) |
           (uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16);
}
// Two e4m3 bytes (the lower 16 bits) to half precision, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n.reg .b16 t;\ncvt.u16.u32 t, %1;\ncvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(two));
    return r;
}
// Four e4m3 bytes to two pairs.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t &lo, uint32_t &hi) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    const uint32_t h = e4m3x2_to_f16x2(two);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace paged
}  // namespace sr
