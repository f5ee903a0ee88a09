// linear.hip -- y = W x for 1 .. 64 token rows against one group-64 affine
// 4-bit matrix (moe_linear): projections and the output head of a decode step
// for several sequences or drafted tokens.
//
// Work: N K / 2 bytes of codes and N K / 16 of scales and biases, each read once,
// 2 T N K operations on the matrix cores.  A weight is dequantised once for all
// T tokens (2.4 vector operations per weight), so up to the widest batch the
// bound is the weight stream, with the dequantisation close behind.
//
// Matrix operands: v_mfma_f32_16x16x32_bf16 with 16 weight rows as A and 16
// tokens as B.  Lane (r = lane & 15, g = lane >> 4) holds row r's codes of columns
// kb + 32 g .. + 31 of a 128-column step (one 16-byte load, 64 contiguous bytes per
// row and instruction), so MFMA j of the step multiplies the columns
// {kb + 32 g + 8 j .. + 7 : g = 0..3}: the sum over k is the same in any order of the
// columns, as long as B holds the same ones.
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kStep = 128;  // columns per wave and step

// One 16-row tile per work group; its KW waves take the 128-column steps in
// turn and their sums meet in LDS in wave order.
template <int NT, int KW>
__global__ __launch_bounds__(KW * 64) void linear_split_kernel(const LinearArgs a) {
    __shared__ f32x4 red[KW > 1 ? KW - 1 : 1][NT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int N = a.N, K = a.K, T = a.T;
    const int row0 = blockIdx.x * 16;
    const size_t row = (size_t)(row0 + r < N ? row0 + r : N - 1);  // clamped, valid
    const uint32_t* qp = a.w.q + row * (size_t)(K / 8);
    const uint16_t* sp = a.w.scale + row * (size_t)(K / kGroup);
    const uint16_t* bp = a.w.bias + row * (size_t)(K / kGroup);
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = wave * kStep; kb < K; kb += KW * kStep) {
        const int k0 = kb + 32 * g;
        const bool live = k0 < K;       // K is a multiple of 64: the last step may be half
        const int kk = live ? k0 : 0;   // clamped, valid
        const u32x4 w = *(const u32x4*)(qp + kk / 8);
        const float s9 = live ? dq_scale(sp[kk / kGroup]) : 0.0f;
        const float b = live ? bf16_to_f32(bp[kk / kGroup]) : 0.0f;
        u32x4 x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int t = 16 * n + r;
            const u32x4* xp = (const u32x4*)(a.x + (size_t)(t < T ? t : T - 1) * K + kk);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[n][j] = xp[j];
                if (!live) x[n][j] = u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 wv = dequant8(w[j], s9, b);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    wv, __builtin_bit_cast(bf16x8, x[n][j]), acc[n], 0, 0, 0);
        }
    }
    if constexpr (KW > 1) {
        if (wave > 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) red[wave - 1][n][lane] = acc[n];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            for (int w = 0; w < KW - 1; ++w) acc[n] += red[w][n][lane];
    }
    // lane (c = lane & 15, g): token 16 n + c, rows row0 + 4 g .. + 3
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = 16 * n + r;
        if (t >= T) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int o = row0 + 4 * g + i;
            if (o >= N) continue;
            if (a.out_bf16) ((uint16_t*)a.y)[(size_t)t * N + o] = f32_to_bf16(acc[n][i]);
            else ((float*)a.y)[(size_t)t * N + o] = acc[n][i];
        }
    }
}

template <int KW>
void launch_split(const LinearArgs& a, hipStream_t s) {
    const dim3 grid((a.N + 15) / 16);
    if (a.T <= 16) linear_split_kernel<1, KW><<<grid, KW * 64, 0, s>>>(a);
    else if (a.T <= 32) linear_split_kernel<2, KW><<<grid, KW * 64, 0, s>>>(a);
    else linear_split_kernel<4, KW><<<grid, KW * 64, 0, s>>>(a);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
    launch_split<4>(a, s);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
