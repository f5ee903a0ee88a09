// e4m3.h -- device helpers of the operators that read or write e4m3 codes with a
// scale per group: the scale and the codes of a group, matrix operands.
#pragma once
#include "q4moe_dev.h"

namespace q4moe {

constexpr int kBlock = 128;  // columns of a scale of the 8-bit products (MOE_E4M3_BLOCK)

// Larger of two magnitudes by bit pattern (a NaN is the largest).
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, float v) {
    const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
    return m > u ? m : u;
}

// Codes of N values (4, 8, ...) of a group whose largest magnitude is amax, and the group's scale:
// scale = amax / 448 and codes of y / scale, both correctly rounded quotients.
template <int N>
__device__ __forceinline__ void e4m3_codes(const float (&y)[N], float amax, float* scale_out, uint32_t (&codes)[N / 4]) {
    float scale, z[N];
    if (amax > 0x1p-70f && amax < 0x1p80f) {
        // Both quotients as products by a reciprocal and their exact remainder: the
        // scale is amax / 448 correctly rounded (checked for every mantissa), and
        // y / scale unless it lies within 2^-22 of a step from the middle of two fp32
        // numbers.
        scale = amax * (1.0f / 448.0f);
        scale = __builtin_fmaf(__builtin_fmaf(-scale, 448.0f, amax), 1.0f / 448.0f, scale);
        const float inv_s = __builtin_amdgcn_rcpf(scale);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = y[i] * inv_s;
            z[i] = __builtin_fmaf(__builtin_fmaf(-t, scale, y[i]), inv_s, t);
        }
    } else {  // where a remainder could leave fp32's range
        scale = amax / 448.0f;  // (0 for the smallest subnormals too)
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = scale == 0.0f ? 0.0f : y[i] / scale;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = z[i] > 448.0f ? 448.0f : z[i] < -448.0f ? -448.0f : z[i];  // (a NaN stays one)
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h], z[4 * h + 1], 0, false);
        codes[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h + 2], z[4 * h + 3], w, true);
    }
    *scale_out = scale;
}

}  // namespace q4moe
