// sort.hip -- token rows into expert order and back (moe_dispatch, moe_combine) and the
// gradients of both (moe_combine_grad; a dispatch's gradient is a combine without weights).
//
//   dispatch       rows[inv[t k + s]] = x[t]             bf16, or e4m3 with a scale per 128 columns
//   combine        y[t] = sum over s of w[t][s] rows[inv[t k + s]] + base[t]
//   combine_grad   d_rows[inv[t k + s]] = w[t][s] dy[t],  d_w[t][s] = <rows[inv[t k + s]], dy[t]>
//
// All three walk tokens: the k rows of a token are found through inv_perm, its own row is
// read or written once, and no two threads write the same piece, so nothing is atomic and
// sums have one order.  They are bound by HBM, for a few tokens by the launch.  A thread holds
// a piece of 8 columns of a token and, with k known when the kernel is compiled, has the pieces
// of all k rows in flight at once.  Indices come from device memory: what is out of range is
// brought into it.
//
// Measured with d = 2048 and k = 8: dispatch of 2048 tokens in e4m3 8 us (43 MB), of 8192 in
// bf16 61 us (5.0 TB/s); combine of 8192 tokens 54 us (6.2 TB/s), its gradient 116 us (4.9 TB/s,
// half of it writes; a copy reaches 5.1), all with outputs that no cache holds; into the buffers of
// the call before 47, 54 and 87.
#include "e4m3.h"
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kThreads = 256;

// The sorted rows of token t's slots.
template <int K>
__device__ __forceinline__ void sorted_rows(const SortArgs& a, int t, size_t (&row)[K]) {
    const int last = a.T * K - 1;
#pragma unroll
    for (int s = 0; s < K; ++s) row[s] = (size_t)min(max(a.inv_perm[(size_t)t * K + s], 0), last);
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

// Thread i of the launch: piece i % pieces of token i / pieces (pieces = a.pieces of a token).
struct Piece {
    int t, c;  // token, first column
    bool live;
};
__device__ __forceinline__ Piece piece_of(const SortArgs& a) {
    const uint32_t i = blockIdx.x * (uint32_t)kThreads + threadIdx.x, p = (uint32_t)a.pieces;
    const uint32_t t = i / p;  // (at most 2^15 tokens of 2^10 pieces)
    Piece r{(int)t, 8 * (int)(i - t * p), t < (uint32_t)a.T};
    if (!r.live) r.t = a.T - 1;  // (a valid one)
    return r;
}

template <int K>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const SortArgs a) {
    const Piece p = piece_of(a);
    if (!p.live) return;
    size_t row[K];
    sorted_rows(a, p.t, row);
    const u32x4 v = *(const u32x4*)(a.x + (size_t)p.t * a.d + p.c);
#pragma unroll
    for (int s = 0; s < K; ++s) *(u32x4*)((uint16_t*)a.rows_out + row[s] * a.d + p.c) = v;
}

// A token has whole groups of 16 lanes (128 columns); the last ones may lie behind the row.
template <int K>
__global__ __launch_bounds__(kThreads) void dispatch_e4m3_kernel(const SortArgs a) {
    Piece p = piece_of(a);
    const int groups = a.pieces / 16;
    p.live = p.live && p.c < a.d;
    size_t row[K];
    sorted_rows(a, p.t, row);
    float f[8];
    unpack8(*(const u32x4*)(a.x + (size_t)p.t * a.d + (p.live ? p.c : 0)), f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_magnitude(m, f[i]);
    if (!p.live) m = 0;
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
    float scale;
    uint32_t w8[2];
    e4m3_codes<8>(f, __uint_as_float(m), &scale, w8);
    if (!p.live) return;
#pragma unroll
    for (int s = 0; s < K; ++s) {
        *(uint2*)((uint8_t*)a.rows_out + row[s] * a.d + p.c) = uint2{w8[0], w8[1]};
        if ((threadIdx.x & 15) == 0) a.scale_out[row[s] * groups + p.c / kBlock] = scale;
    }
}

// Sixteen bytes; ONCE: not kept in the caches for others.
template <bool ONCE>
__device__ __forceinline__ u32x4 load16(const void* p) {
    if constexpr (ONCE) return __builtin_nontemporal_load((const u32x4*)p);
    else return *(const u32x4*)p;
}

template <int K, bool ONCE>
__global__ __launch_bounds__(kThreads) void combine_kernel(const SortArgs a) {
    const Piece p = piece_of(a);
    if (!p.live) return;
    size_t row[K];
    sorted_rows(a, p.t, row);
    u32x4 v[K];
    float w[K];
#pragma unroll
    for (int s = 0; s < K; ++s) {
        v[s] = load16<ONCE>(a.rows + row[s] * a.d + p.c);
        w[s] = a.w ? a.w[(size_t)p.t * K + s] : 1.0f;
    }
    const size_t at = (size_t)p.t * a.d + p.c;
    u32x4 b = {0u, 0u, 0u, 0u};
    if (a.base) b = *(const u32x4*)(a.base + at);
    float sum[8], f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
#pragma unroll
    for (int s = 0; s < K; ++s) {
        unpack8(v[s], f);
        if (w[s] != 0.0f) {  // (a slot of weight 0 counts for nothing, whatever its row holds)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[s], f[i], sum[i]);
        }
    }
    if (a.base) {
        unpack8(b, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += f[i];
    }
    *(u32x4*)(a.y + at) = pack8(sum);
}

// One piece of a token's gradients: d_rows of all slots, and what the piece adds to d_w.
template <int K, bool ONCE>
__device__ __forceinline__ void grad_piece(const SortArgs& a, int t, int c, const size_t (&row)[K],
                                           const float (&w)[K], float (&dot)[K]) {
    u32x4 v[K];
    float dy[8], f[8];
#pragma unroll
    for (int s = 0; s < K; ++s) v[s] = load16<ONCE>(a.rows + row[s] * a.d + c);
    unpack8(load16<ONCE>(a.dy + (size_t)t * a.d + c), dy);
#pragma unroll
    for (int s = 0; s < K; ++s) {
        unpack8(v[s], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[s] = __builtin_fmaf(f[i], dy[i], dot[s]);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = w[s] * dy[i];
        *(u32x4*)((uint16_t*)a.rows_out + row[s] * a.d + c) = pack8(f);
    }
}

// d_w of a slot of weight w whose row and dy have the sum v: a slot of weight 0 counts for nothing,
// so what its row holds (nothing that was ever written, say) makes no NaN or infinity here.
__device__ __forceinline__ float weight_grad(float w, float v) {
    return w == 0.0f && !__builtin_isfinite(v) ? 0.0f : v;
}

// Rows of up to 8 G columns: G lanes a token.
template <int K, int G>
__global__ __launch_bounds__(kThreads) void combine_grad_short_kernel(const SortArgs a) {
    const int t0 = (int)((blockIdx.x * kThreads + threadIdx.x) / G), lane = threadIdx.x & (G - 1);
    const int t = min(t0, a.T - 1);
    size_t row[K];
    sorted_rows(a, t, row);
    float w[K], dot[K];
#pragma unroll
    for (int s = 0; s < K; ++s) {
        w[s] = a.w[(size_t)t * K + s];
        dot[s] = 0.0f;
    }
    if (t0 < a.T && 8 * lane < a.d) grad_piece<K, false>(a, t, 8 * lane, row, w, dot);
#pragma unroll
    for (int s = 0; s < K; ++s) {
        const float v = group_sum<G>(dot[s]);
        if (lane == 0 && t0 < a.T) a.d_w[(size_t)t * K + s] = weight_grad(w[s], v);
    }
}

// A work group a token.
template <int K, bool ONCE>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(const SortArgs a) {
    __shared__ float part[K][kThreads / 64];
    const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    size_t row[K];
    sorted_rows(a, t, row);
    float w[K], dot[K];
#pragma unroll
    for (int s = 0; s < K; ++s) {
        w[s] = a.w[(size_t)t * K + s];
        dot[s] = 0.0f;
    }
    for (int c = 8 * (int)threadIdx.x; c < a.d; c += 8 * kThreads) grad_piece<K, ONCE>(a, t, c, row, w, dot);
#pragma unroll
    for (int s = 0; s < K; ++s) {
        const float v = wave_sum_dpp(dot[s]);
        if (lane == 0) part[s][wave] = v;
    }
    __syncthreads();
    if (threadIdx.x < K) {
        float v = part[threadIdx.x][0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) v += part[threadIdx.x][i];
        const size_t at = (size_t)t * K + threadIdx.x;
        a.d_w[at] = weight_grad(a.w[at], v);
    }
}

template <int N>
struct Int {
    static constexpr int value = N;
};

// f(Int<k>) for the k of the call.
template <typename F>
void with_k(int k, F f) {
    switch (k) {
        case 1: return f(Int<1>{});
        case 2: return f(Int<2>{});
        case 3: return f(Int<3>{});
        case 4: return f(Int<4>{});
        case 5: return f(Int<5>{});
        case 6: return f(Int<6>{});
        case 7: return f(Int<7>{});
        default: return f(Int<8>{});
    }
}
static_assert(MOE_MAX_TOPK == 8, "with_k");

// Expert rows that the last-level cache does not hold: loads that ask not to be kept leave it to the
// stores (d = 2048, k = 8, us with and without: combine of 2048 tokens 16.0 and 14.4, of 3200 23.1
// and 25.6, of 8192 54 and 65; its gradient of 3200 38 and 38, of 8192 116 and 116, into the buffer of
// the call before 87 and 110.  Stores that ask for it too: 111, and 106 into that buffer, so they
// do not).
bool read_once(const SortArgs& a) { return 2LL * a.T * a.k * a.d >= 96LL << 20; }

unsigned blocks_for(long long threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }

}  // namespace

hipError_t launch_dispatch(const SortArgs& a0, hipStream_t s) {
    SortArgs a = a0;
    a.pieces = a.scale_out ? (a.d + kBlock - 1) / kBlock * 16 : a.d / 8;
    const unsigned n = blocks_for((long long)a.T * a.pieces);
    with_k(a.k, [&](auto k) {
        if (a.scale_out) dispatch_e4m3_kernel<decltype(k)::value><<<n, kThreads, 0, s>>>(a);
        else dispatch_kernel<decltype(k)::value><<<n, kThreads, 0, s>>>(a);
    });
    trace_point(s);
    return hipGetLastError();
}

hipError_t launch_combine(const SortArgs& a0, hipStream_t s) {
    SortArgs a = a0;
    a.pieces = a.d / 8;
    const unsigned n = blocks_for((long long)a.T * a.pieces);
    const bool once = read_once(a);
    with_k(a.k, [&](auto k) {
        if (once) combine_kernel<decltype(k)::value, true><<<n, kThreads, 0, s>>>(a);
        else combine_kernel<decltype(k)::value, false><<<n, kThreads, 0, s>>>(a);
    });
    trace_point(s);
    return hipGetLastError();
}

// Rows of up to 512 columns share work groups (30000 tokens of 192 columns, k = 8: 59 us with a
// work group each).
hipError_t launch_combine_grad(const SortArgs& a, hipStream_t s) {
    const bool once = read_once(a);
    with_k(a.k, [&](auto k) {
        constexpr int K = decltype(k)::value;
        if (a.d <= 64) combine_grad_short_kernel<K, 8><<<blocks_for(8LL * a.T), kThreads, 0, s>>>(a);
        else if (a.d <= 128) combine_grad_short_kernel<K, 16><<<blocks_for(16LL * a.T), kThreads, 0, s>>>(a);
        else if (a.d <= 256) combine_grad_short_kernel<K, 32><<<blocks_for(32LL * a.T), kThreads, 0, s>>>(a);
        else if (a.d <= 512) combine_grad_short_kernel<K, 64><<<blocks_for(64LL * a.T), kThreads, 0, s>>>(a);
        else if (once) combine_grad_kernel<K, true><<<a.T, kThreads, 0, s>>>(a);
        else combine_grad_kernel<K, false><<<a.T, kThreads, 0, s>>>(a);
    });
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
