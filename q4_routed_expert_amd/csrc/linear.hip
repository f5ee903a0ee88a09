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
//
// Two kernels.  Both add a row's products in the same order whatever T is: which of
// them runs, and how it splits K, follows from N and K alone.
//   linear_split_kernel   few rows: one 16-row tile per work group, its waves share K
//                         and their sums meet in LDS (otherwise most CUs would idle)
//   linear_stream_kernel  many rows: every wave owns its tiles; x goes through LDS in
//                         chunks of K, in operand order, for all waves of the group
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kStep = 128;  // columns per wave and step

// D of the 16x16 product: lane (c = lane & 15, g) holds token 16 n + c, rows
// row0 + 4 g .. + 3.
template <int NT>
__device__ __forceinline__ void store_tile(const LinearArgs& a, const f32x4 (&acc)[NT], int row0, int lane) {
    const int c = lane & 15, o = row0 + 4 * (lane >> 4);
    const int N = a.N;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = 16 * n + c;
        if (t >= a.T) continue;
        const size_t at = (size_t)t * N + o;
        if (o + 4 <= N && (N & 3) == 0) {  // four neighbours, aligned
            if (a.out_bf16)
                *(uint2*)((uint16_t*)a.y + at) = uint2{pack_bf16x2(acc[n][0], acc[n][1]), pack_bf16x2(acc[n][2], acc[n][3])};
            else
                *(f32x4*)((float*)a.y + at) = acc[n];
            continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (o + i >= N) break;
            if (a.out_bf16) ((uint16_t*)a.y)[at + i] = f32_to_bf16(acc[n][i]);
            else ((float*)a.y)[at + i] = acc[n][i];
        }
    }
}

// One 16-row tile per work group; its KW waves take the 128-column steps in
// turn and their sums meet in LDS in wave order.
template <int NT, int KW>
__global__ __launch_bounds__(KW * 64) void linear_split_kernel(const LinearArgs a) {
    __shared__ f32x4 red[KW - 1][NT][64];
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
    if (wave > 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) red[wave - 1][n][lane] = acc[n];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        for (int w = 0; w < KW - 1; ++w) acc[n] += red[w][n][lane];
    store_tile<NT>(a, acc, row0, lane);
}

// Many rows.  x lies in LDS in operand order, [step][j][n][g][token] of 16 bytes, so that
// a wave's read of one operand is contiguous; NB is the number of tokens it has room for
// (8: lanes of tokens 8 .. 15 read those of 0 .. 7 again, their results are not stored).
//   RES    all of x (NB K 2 <= 128 KB) is staged once; after that the waves run without
//          barriers, each over its own tiles (wave w of group b: tiles w G + b, then every
//          16 G, so that any number of tiles spreads over the CUs)
//   else   one 512-column chunk of x at a time, double buffered, a barrier per chunk; a
//          work group's waves take neighbouring tiles
// The grid is one work group per CU; the next chunk's weights, across tiles too, are
// loaded before the current chunk's products.
//   VEC    K is a multiple of 512: a chunk's eight scales of a row are one aligned load
constexpr int kChunk = 512;
constexpr int kSteps = kChunk / kStep;
constexpr int kCus = 256;

template <int NB, int WAVES, bool RES, bool VEC>
__global__ __launch_bounds__(WAVES * 64) void linear_stream_kernel(const LinearArgs a) {
    constexpr int NT = (NB + 15) / 16, TB = NB < 16 ? NB : 16, THREADS = WAVES * 64;
    constexpr int kStepPieces = NB * 16, kChunkPieces = NB * 64;
    constexpr int XP = RES ? 1 : kChunkPieces / THREADS;  // pieces of a chunk per thread
    __shared__ u32x4 s_x[RES ? 8192 : 2 * kChunkPieces];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int N = a.N, K = a.K, T = a.T, G = gridDim.x;
    // neighbouring units go to work groups of one XCD (group i runs on XCD i % 8), whose L2
    // joins the half lines that two tiles write
    const int b = (int)blockIdx.x, me = G % 8 == 0 ? (b & 7) * (G / 8) + (b >> 3) : b;
    // piece (token t, columns 8 c .. + 7) of x, 0 past the end; its place in a chunk or x
    auto x_piece = [&](int t, int col) {
        const bool live = t < T && col < K;
        const u32x4 v = *(const u32x4*)(a.x + (live ? (size_t)t * K + col : 0));
        return live ? v : u32x4{0u, 0u, 0u, 0u};
    };
    auto x_place = [&](int t, int c) {  // columns 128 (c >> 4) + 32 gg + 8 j
        const int gg = (c >> 2) & 3, j = c & 3;
        return (c >> 4) * kStepPieces + ((j * NT + (t >> 4)) * 4 + gg) * TB + (t & (TB - 1));
    };
    struct Weights {
        u32x4 q[kSteps];
        u32x4 s, b;                       // VEC: the chunk's eight scales, biases
        uint16_t s1[kSteps], b1[kSteps];  // else: this lane's of each step
    };
    const int unit_rows = RES ? 16 : 16 * WAVES;
    const int units = (N + unit_rows - 1) / unit_rows, stride = RES ? WAVES * G : G;
    auto row_of = [&](int u) { return RES ? u * 16 : (u * WAVES + wave) * 16; };
    auto load = [&](Weights& v, int u, int kc) {
        const int row0 = row_of(u) + r;
        const size_t row = (size_t)(row0 < N ? row0 : N - 1);  // clamped, valid
        const uint32_t* qp = a.w.q + row * (size_t)(K / 8);
        const size_t so = row * (size_t)(K / kGroup);
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            const int k0 = kc + st * kStep + 32 * g, kk = VEC || k0 < K ? k0 : 0;  // clamped, valid
            v.q[st] = *(const u32x4*)(qp + kk / 8);
            if constexpr (!VEC) {
                v.s1[st] = a.w.scale[so + kk / kGroup];
                v.b1[st] = a.w.bias[so + kk / kGroup];
            }
        }
        if constexpr (VEC) {
            v.s = *(const u32x4*)(a.w.scale + so + kc / kGroup);
            v.b = *(const u32x4*)(a.w.bias + so + kc / kGroup);
        }
    };
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // One chunk.  The operands of x for product q + 1 are read before the weights of
    // product q are dequantised, so that their latency runs under that.
    auto products = [&](const Weights& v, const u32x4* x, int kc) {
        const u32x4* xl = x + g * TB + (r & (TB - 1));
        const int steps = VEC ? kSteps : min(kSteps, (K - kc + kStep - 1) / kStep);
        u32x4 xo[2][NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) xo[0][n] = xl[n * 4 * TB];
        float s9 = 0.0f, bi = 0.0f;
#pragma unroll
        for (int q = 0; q < 4 * kSteps; ++q) {
            const int st = q >> 2, j = q & 3;
            if (!VEC && st >= steps) break;  // uniform
            if (q + 1 < 4 * kSteps && (VEC || j < 3 || st + 1 < steps)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    xo[(q + 1) & 1][n] = xl[((q + 1) >> 2) * kStepPieces + (((q + 1) & 3) * NT + n) * 4 * TB];
            }
            __builtin_amdgcn_sched_barrier(0);
            if (j == 0) {
                if constexpr (VEC) {  // group 2 st + (g >> 1): one half of word st
                    const int up = g & 2 ? 0 : 16;
                    s9 = __uint_as_float((v.s[st] << up) & 0xFFFF0000u) * 512.0f;
                    bi = __uint_as_float((v.b[st] << up) & 0xFFFF0000u);
                } else {
                    const bool live = kc + st * kStep + 32 * g < K;
                    s9 = live ? dq_scale(v.s1[st]) : 0.0f;
                    bi = live ? bf16_to_f32(v.b1[st]) : 0.0f;
                }
            }
            const bf16x8 wv = dequant8(v.q[st][j], s9, bi);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, xo[q & 1][n]),
                                                                 acc[n], 0, 0, 0);
        }
    };
    int u = RES ? wave * G + me : me, kc = 0, buf = 0;
    Weights w0, w1;
    if (u < units) load(w0, u, 0);
    if constexpr (RES) {
        const int per = (K + kStep - 1) / kStep * 16;  // pieces per token
        for (int i = tid; i < NB * per; i += THREADS) {
            const int t = i / per, c = i - t * per;
            s_x[x_place(t, c)] = x_piece(t, 8 * c);
        }
    } else {
#pragma unroll
        for (int p = 0; p < XP; ++p) {
            const int i = tid + p * THREADS, t = i >> 6, c = i & 63;
            s_x[x_place(t, c)] = x_piece(t, 8 * c);
        }
    }
    __syncthreads();
    // one chunk with `cur` while `nxt` is loaded
    auto chunk = [&](const Weights& cur, Weights& nxt) {
        const bool last = kc + kChunk >= K;
        const int u2 = last ? u + stride : u, kc2 = last ? 0 : kc + kChunk;
        const bool more = u2 < units;
        u32x4 xn[XP];
        if (more) {
            load(nxt, u2, kc2);
            if constexpr (!RES) {
#pragma unroll
                for (int p = 0; p < XP; ++p) {
                    const int i = tid + p * THREADS;
                    xn[p] = x_piece(i >> 6, kc2 + 8 * (i & 63));
                }
            }
        }
        products(cur, RES ? s_x + kc / kStep * kStepPieces : s_x + buf * kChunkPieces, kc);
        if (last) {
            store_tile<NT>(a, acc, row_of(u), lane);
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        if constexpr (!RES) {
            if (more) {
                buf ^= 1;  // (read last before the previous barrier)
#pragma unroll
                for (int p = 0; p < XP; ++p) {
                    const int i = tid + p * THREADS;
                    s_x[buf * kChunkPieces + x_place(i >> 6, i & 63)] = xn[p];
                }
                __syncthreads();
            }
        }
        u = u2;
        kc = kc2;
    };
    while (u < units) {  // (u: by wave with RES, by work group else)
        chunk(w0, w1);
        if (u >= units) break;
        chunk(w1, w0);
    }
}

template <int NB, bool RES>
void launch_stream(const LinearArgs& a, hipStream_t s) {
    constexpr int WAVES = RES ? 16 : 8;
    const int tiles = (a.N + 15) / 16, units = RES ? tiles : (tiles + WAVES - 1) / WAVES;
    const int grid = units < kCus ? units : kCus;
    if (a.K % kChunk == 0) linear_stream_kernel<NB, WAVES, RES, true><<<grid, WAVES * 64, 0, s>>>(a);
    else linear_stream_kernel<NB, WAVES, RES, false><<<grid, WAVES * 64, 0, s>>>(a);
}

template <int NB>
void launch(const LinearArgs& a, hipStream_t s) {
    if (a.N < 16384) linear_split_kernel<(NB + 15) / 16, 4><<<(a.N + 15) / 16, 256, 0, s>>>(a);
    else if (NB * ((a.K + kStep - 1) / kStep) <= 512) launch_stream<NB, true>(a, s);
    else if constexpr (NB > 8) launch_stream<NB, false>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
    if (a.T <= 8) launch<8>(a, s);
    else if (a.T <= 16) launch<16>(a, s);
    else if (a.T <= 32) launch<32>(a, s);
    else launch<64>(a, s);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
