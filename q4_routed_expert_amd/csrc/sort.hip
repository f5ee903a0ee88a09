// sort.hip -- token rows into expert order and back (moe_dispatch, moe_combine) and the
// gradients of both (moe_combine_grad; a dispatch's gradient is a combine without weights).
//
//   dispatch       rows[inv[t k + s]] = x[t]             bf16, or e4m3 with a scale per 128 columns
//   combine        y[t] = sum over s of w[t][s] rows[inv[t k + s]] + base[t]
//   combine_grad   d_rows[inv[t k + s]] = w[t][s] dy[t],  d_w[t][s] = <rows[inv[t k + s]], dy[t]>
//
// All three walk tokens: the k rows of a token are found through inv_perm, its own row is
// read or written once, and no two work groups write the same row, so nothing is atomic and
// sums have one order.  They are bound by HBM (rows of d columns are contiguous), for a few
// tokens by the launch.  Indices come from device memory: what is out of range is brought
// into it.
#include "e4m3.h"
#include "ops.h"

namespace q4moe {
namespace {

// Most threads of a token; a thread holds pieces of 8 columns: piece j of thread t covers
// columns 8 (t + threads j) .. + 7.
constexpr int kMaxThreads = 256;

__device__ __forceinline__ size_t sorted_row(const SortArgs& a, int t, int s) {
    const int n = a.T * a.k;
    return (size_t)min(max(a.inv_perm[(size_t)t * a.k + s], 0), n - 1);
}

__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return v;
}

template <bool E4M3>
__global__ __launch_bounds__(kMaxThreads) void dispatch_kernel(const SortArgs a) {
    const int t = blockIdx.x, d = a.d, k = a.k, groups = (d + kBlock - 1) / kBlock;
    // whole waves stay: lanes behind the row take part in the group's maximum
    for (int c0 = 0; c0 < d; c0 += 8 * blockDim.x) {
        const int c = c0 + 8 * (int)threadIdx.x;
        const bool live = c < d;
        const u32x4 v = *(const u32x4*)(a.x + (size_t)t * d + (live ? c : 0));
        if constexpr (!E4M3) {
            if (live)
                for (int s = 0; s < k; ++s) *(u32x4*)((uint16_t*)a.rows_out + sorted_row(a, t, s) * d + c) = v;
        } else {
            float f[8];
            unpack8(v, f);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max_magnitude(m, f[i]);
            if (!live) m = 0;
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
            float scale;
            uint32_t w8[2];
            e4m3_codes<8>(f, __uint_as_float(m), &scale, w8);
            if (live)
                for (int s = 0; s < k; ++s) {
                    const size_t row = sorted_row(a, t, s);
                    *(uint2*)((uint8_t*)a.rows_out + row * d + c) = uint2{w8[0], w8[1]};
                    if ((threadIdx.x & 15) == 0) a.scale_out[row * groups + c / kBlock] = scale;
                }
        }
    }
}

__global__ __launch_bounds__(kMaxThreads) void combine_kernel(const SortArgs a) {
    const int t = blockIdx.x, d = a.d, k = a.k;
    const int c = 8 * ((int)blockIdx.y * (int)blockDim.x + (int)threadIdx.x);
    if (c >= d) return;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    for (int s = 0; s < k; ++s) {
        const float w = a.w ? a.w[(size_t)t * k + s] : 1.0f;
        float f[8];
        unpack8(*(const u32x4*)(a.rows + sorted_row(a, t, s) * d + c), f);
        if (w != 0.0f) {  // (a slot of weight 0 counts for nothing, whatever its row holds)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w, f[i], sum[i]);
        }
    }
    if (a.base) {
        float f[8];
        unpack8(*(const u32x4*)(a.base + (size_t)t * d + c), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += f[i];
    }
    *(u32x4*)(a.y + (size_t)t * d + c) = pack8(sum);
}

__global__ __launch_bounds__(kMaxThreads) void combine_grad_kernel(const SortArgs a) {
    __shared__ float part[MOE_MAX_TOPK][kMaxThreads / 64];
    const int t = blockIdx.x, d = a.d, k = a.k;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    float dot[MOE_MAX_TOPK];
#pragma unroll
    for (int s = 0; s < MOE_MAX_TOPK; ++s) dot[s] = 0.0f;
    for (int c = 8 * (int)threadIdx.x; c < d; c += 8 * blockDim.x) {
        float dy[8];
        unpack8(*(const u32x4*)(a.dy + (size_t)t * d + c), dy);
#pragma unroll
        for (int s = 0; s < MOE_MAX_TOPK; ++s) {
            if (s >= k) break;
            const size_t at = sorted_row(a, t, s) * d + c;
            float f[8];
            unpack8(*(const u32x4*)(a.rows + at), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[s] = __builtin_fmaf(f[i], dy[i], dot[s]);
            if (a.rows_out) {
                const float w = a.w[(size_t)t * k + s];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = w * dy[i];
                *(u32x4*)((uint16_t*)a.rows_out + at) = pack8(f);
            }
        }
    }
    if (!a.d_w) return;
#pragma unroll
    for (int s = 0; s < MOE_MAX_TOPK; ++s) {
        const float v = wave_sum_dpp(dot[s]);
        if (lane == 0) part[s][wave] = v;
    }
    __syncthreads();
    if ((int)threadIdx.x < k) {
        float v = part[threadIdx.x][0];
        for (int w = 1; w < waves; ++w) v += part[threadIdx.x][w];
        a.d_w[(size_t)t * k + threadIdx.x] = v;
    }
}

int threads_for(int d) {
    const int n = (d / 8 + 63) / 64 * 64;
    return n < kMaxThreads ? n : kMaxThreads;
}

}  // namespace

hipError_t launch_dispatch(const SortArgs& a, hipStream_t s) {
    if (a.scale_out) dispatch_kernel<true><<<a.T, threads_for(a.d), 0, s>>>(a);
    else dispatch_kernel<false><<<a.T, threads_for(a.d), 0, s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

hipError_t launch_combine(const SortArgs& a, hipStream_t s) {
    const int n = threads_for(a.d);
    combine_kernel<<<dim3(a.T, (a.d / 8 + n - 1) / n), n, 0, s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

hipError_t launch_combine_grad(const SortArgs& a, hipStream_t s) {
    combine_grad_kernel<<<a.T, threads_for(a.d), 0, s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
