// norm.hip -- residual addition and root-mean-square norm of token rows.
//
//   r = x + residual                 (fp32 sum, rounded once to the residual's type, stored)
//   y = r / sqrt(mean(r^2) + eps) * w
//
// in fp32 from the stored r, rounded once to bf16; or, per 64 columns, to e4m3
// codes of y / scale with the fp32 scale max|y| / 448 (448 = the largest e4m3
// value), from the unrounded y.  The quotient is by the scale that is stored: a
// factor 448 / max|y| rounds otherwise (one code in 10^5 lands on the other side of a
// border) and leaves fp32's range for a small max|y|.
//
// Every input is read once and every output written once: a row stays in the
// registers between its sum of squares and its scaling.  The kernel is bound by
// HBM for long chunks and by the launch for a few tokens.
#include "ops.h"

namespace q4moe {
namespace {

// One row per W waves; a lane holds NV pieces of 8 columns: piece j of thread
// t covers columns 8 (t + 64 W j) .. + 7, so a 64-column group is eight
// neighbouring lanes.
template <int W, int NV, bool RES, bool F32>
__global__ __launch_bounds__(W * 64) void add_norm_kernel(const NormArgs a) {
    __shared__ float s_sum[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int d = a.d;
    const size_t row = (size_t)blockIdx.x * (size_t)d;
    float v[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + 64 * W * j);
        const bool live = c < d;
        const size_t o = row + (live ? c : 0);  // clamped, always valid
        const u32x4 xv = *(const u32x4*)(a.x + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[j][2 * i] = __uint_as_float(xv[i] << 16);
            v[j][2 * i + 1] = __uint_as_float(xv[i] & 0xFFFF0000u);
        }
        if constexpr (RES) {
            if constexpr (F32) {
                const float* rp = (const float*)a.residual + o;
                const f32x4 r0 = ((const f32x4*)rp)[0], r1 = ((const f32x4*)rp)[1];
                f32x4 o0, o1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[j][i] += r0[i];
                    v[j][4 + i] += r1[i];
                    o0[i] = v[j][i];
                    o1[i] = v[j][4 + i];
                }
                if (live && a.residual_out) {
                    f32x4* op = (f32x4*)((float*)a.residual_out + o);
                    op[0] = o0;
                    op[1] = o1;
                }
            } else {
                const u32x4 rv = *(const u32x4*)((const uint16_t*)a.residual + o);
                u32x4 ov;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ov[i] = pack_bf16x2(v[j][2 * i] + __uint_as_float(rv[i] << 16),
                                        v[j][2 * i + 1] + __uint_as_float(rv[i] & 0xFFFF0000u));
                    // the norm sees the residual as it is stored
                    v[j][2 * i] = __uint_as_float(ov[i] << 16);
                    v[j][2 * i + 1] = __uint_as_float(ov[i] & 0xFFFF0000u);
                }
                if (live && a.residual_out) *(u32x4*)((uint16_t*)a.residual_out + o) = ov;
            }
        }
        float p = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) p += v[j][i] * v[j][i];
        ss += live ? p : 0.0f;
    }
    ss = wave_sum_dpp(ss);
    if constexpr (W > 1) {
        if (lane == 0) s_sum[wave] = ss;
        __syncthreads();
        ss = s_sum[0];
#pragma unroll
        for (int w = 1; w < W; ++w) ss += s_sum[w];
    }
    const float inv = rsqrtf(ss / (float)d + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + 64 * W * j);
        const bool live = c < d;
        const u32x4 wv = *(const u32x4*)(a.weight + (live ? c : 0));
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = v[j][2 * i] * inv * (__uint_as_float(wv[i] << 16) + a.w_add);
            y[2 * i + 1] = v[j][2 * i + 1] * inv * (__uint_as_float(wv[i] & 0xFFFF0000u) + a.w_add);
        }
        if (a.y) {
            u32x4 yv;
#pragma unroll
            for (int i = 0; i < 4; ++i) yv[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
            if (live) *(u32x4*)(a.y + row + c) = yv;
        }
        if (a.y8) {
            // largest magnitude of the 64-column group, by bit pattern (a NaN is the largest)
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
            const float amax = __uint_as_float(m);
            float scale, z[8];
            if (amax > 0x1p-70f && amax < 0x1p80f) {
                // Both quotients as products by a reciprocal and their exact remainder: the
                // scale is amax / 448 correctly rounded (checked for every mantissa), and
                // y / scale unless it lies within 2^-22 of a step from the middle of two fp32
                // numbers.  (2048 x 2048 with eight IEEE divisions: 8.6 us instead of 7.7.)
                scale = amax * (1.0f / 448.0f);
                scale = __builtin_fmaf(__builtin_fmaf(-scale, 448.0f, amax), 1.0f / 448.0f, scale);
                const float inv_s = __builtin_amdgcn_rcpf(scale);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float t = y[i] * inv_s;
                    z[i] = __builtin_fmaf(__builtin_fmaf(-t, scale, y[i]), inv_s, t);
                }
            } else {  // where a remainder could leave fp32's range
                scale = amax / 448.0f;  // (0 for the smallest subnormals too)
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = scale == 0.0f ? 0.0f : y[i] / scale;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = z[i] > 448.0f ? 448.0f : z[i] < -448.0f ? -448.0f : z[i];  // (a NaN stays one)
            uint32_t w8[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int w = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h], z[4 * h + 1], 0, false);
                w8[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h + 2], z[4 * h + 3], w, true);
            }
            if (live) {
                *(uint2*)(a.y8 + row + c) = uint2{w8[0], w8[1]};
                if ((tid & 7) == 0) a.y8_scale[(row + c) / kGroup] = scale;
            }
        }
    }
}

template <int W, int NV>
void launch(const NormArgs& a, hipStream_t s) {
    if (!a.residual) add_norm_kernel<W, NV, false, false><<<a.T, W * 64, 0, s>>>(a);
    else if (a.res_f32) add_norm_kernel<W, NV, true, true><<<a.T, W * 64, 0, s>>>(a);
    else add_norm_kernel<W, NV, true, false><<<a.T, W * 64, 0, s>>>(a);
}

}  // namespace

// As many waves a row as have a piece of 8 columns for most of their lanes: 32768 rows
// with a bf16 residual take, for 512 columns, 24.1 us with one wave, 25.2 with two and
// 36.2 with four; for 576 / 1024 28.8 / 46.2 with two and 39.9 / 47.4 with four (one wave
// with two pieces a lane: 32.2 / 48.5); for 1088 / 2048 50.9 / 90.8 with four, 53.5 / 93.1
// with two.  One row: 1.9 us in every form, but 2.3 to 3.0 with more than one piece.
// 32768 rows of 2048 with an fp32 residual move 805 MB in 138 us, 5.8 TB/s.
hipError_t launch_add_norm(const NormArgs& a, hipStream_t s) {
    if (a.d <= 512) launch<1, 1>(a, s);
    else if (a.d <= 1024) launch<2, 1>(a, s);
    else if (a.d <= 2048) launch<4, 1>(a, s);
    else if (a.d <= 4096) launch<4, 2>(a, s);
    else launch<4, 4>(a, s);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
