// What the kernels of attention over the paged 8-bit cache share.
#pragma once

#include <cuda.h>

#include "paged.cuh"
#include "tc.cuh"

namespace sr {
namespace paged {

struct AttnParams {
    const __nv_bfloat16 *q;
    long long q_stride;  // elements from token to token
    const int32_t *cu, *kv_lens, *table;
    const float *k_scale, *v_scale;
    __nv_bfloat16 *o;
    float *lse;  // may be null
    uint32_t *status;
    int *tickets;     // zero at the start of a call
    float *parts;     // partial O
    float2 *part_ml;  // their m and l
    float scale_log2; // scale log2(e)
    int n_seqs, total, max_len, max_kv, h_q, h_kv, group, page, n_pages, max_pages;
};

// CTAs of the few-rows kernel: one per SM.
constexpr int kRowsMaxCtas = 148;

constexpr float kNone = -1e30f;  // m of a row that has seen nothing
constexpr float kSlack = 4.f;    // growth of the maximum that m does not follow
constexpr float kShift = 11.f;   // weights are at most 2^(kShift + kSlack) = 2^15

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Power of two that brings a row whose largest element is `top` to at most 1.
__device__ __forceinline__ float row_down(float top) {
    if (!(top > 0.f) || top > 3.402823466e38f) return 1.f;
    int e;
    frexpf(top, &e);
    return ldexpf(1.f, -min(max(e, -100), 120));
}
// A block's scale, within the range that sr_kv_append writes; NaN becomes the least.
__device__ __forceinline__ float usable_scale(float s) { return fminf(fmaxf(s, 0x1p-32f), 0x1p32f); }
// log(sum exp(s)) of a row from its base-2 m and l.
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.f ? -INFINITY : 0.69314718055994531f * (m - kShift + log2f(l));
}
// e4m3 NaN bytes (0x7f, 0xff) of a word.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ bool has_nan(uint32_t w) { return nan_bits(w) != 0; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_bits(w) >> 7) * 0xffu); }

cudaError_t attend_rows(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int d, cudaStream_t st);

}  // namespace paged
}  // namespace sr
