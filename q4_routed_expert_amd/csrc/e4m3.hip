// e4m3.hip -- products of e4m3 rows with e4m3 matrices, one scale per token and 128
// columns of x and one per 128 x 128 block of W (moe_linear_scaled, moe_experts_scaled):
//
//   y[t][n] = sum over blocks b of xs[t][b] ws[n / 128][b] sum over k in b of x[t][k] w[n][k]
//
// Codes become bf16 on the way into the matrix cores (exactly: 4 significant bits, exponents
// -9 .. 8), four v_mfma_f32_16x16x32_bf16 per block with 16 weight rows as A and 16 tokens
// as B; then the block's fp32 sum is scaled and added by four fused multiply-adds.  The matrix
// cores' own e4m3 products are twice as fast, but they cut every product to 13 bits below the
// largest of its group of columns: sums of 128 normally distributed values came out
// 1.5e-5 off (2-norm), through bf16 9e-9.
// A block's sum is the same in any order of its columns, as long as A and B hold the same
// ones: lane (r = lane & 15, g = lane >> 4) holds columns 32 g .. + 31 of row r of both.  In D
// lane (c, g) holds token c, weight rows 4 g .. + 3, so a lane's factor xs * ws is one number
// per 16 tokens and block.
//
// Gated output: the matrix holds gate and up rows; a wave computes 16 rows of each, so both
// sums of a column are in one lane, and silu(gate) * up leaves in e4m3.
#include "e4m3.h"
#include "ops.h"

namespace q4moe {
namespace {

// What a work group's rows are: rows row0 .. row0 + n - 1 of x and y, matrix e.
struct RowSpan {
    int row0, n, e;
};

// Tile j of TR rows: of the rows themselves, or of the map of expert-sorted rows.  Map
// entries come from device memory: what is out of range is brought into it.
template <int TR>
__device__ __forceinline__ RowSpan span_of(const ProductArgs& a, int j) {
    RowSpan s{0, 0, 0};
    if (!a.map) {
        s.row0 = j * TR;
        s.n = a.rows - s.row0;
    } else {
        if (j >= *a.n_map) return s;
        s.e = min(max(a.map[2 * j], 0), a.E - 1);
        s.row0 = min(max(a.map[2 * j + 1], 0), a.rows);
        s.n = min(a.offsets[s.e + 1], a.rows) - s.row0;
    }
    s.n = min(max(s.n, 0), TR);
    return s;
}

// 32 codes of a row as four bf16 operands.
struct Operand {
    bf16x8 v[4];
};

__device__ __forceinline__ uint32_t two_bf16(uint32_t codes, bool high) {
    return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)codes, 1.0f, true))
                : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)codes, 1.0f, false));
}

__device__ __forceinline__ Operand operand(const u32x4& lo, const u32x4& hi) {
    Operand o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = j < 2 ? lo[2 * j] : hi[2 * j - 4], b = j < 2 ? lo[2 * j + 1] : hi[2 * j - 3];
        o.v[j] = __builtin_bit_cast(bf16x8, u32x4{two_bf16(a, false), two_bf16(a, true), two_bf16(b, false),
                                                  two_bf16(b, true)});
    }
    return o;
}

__device__ __forceinline__ f32x4 block_product(const Operand& w, const Operand& x) {
    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[j], x.v[j], d, 0, 0, 0);
    return d;
}

// Four sums of one token, weight rows o .. o + 3.
__device__ __forceinline__ void store4(const ProductArgs& a, size_t row, int o, const f32x4& v) {
    const size_t at = row * (size_t)a.N + o;
    if (o + 4 <= a.N && (a.N & 3) == 0) {  // four neighbours, aligned
        if (a.out_bf16)
            *(uint2*)((uint16_t*)a.y + at) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
            *(f32x4*)((float*)a.y + at) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (o + i >= a.N) break;
        if (a.out_bf16) ((uint16_t*)a.y)[at + i] = f32_to_bf16(v[i]);
        else ((float*)a.y)[at + i] = v[i];
    }
}

constexpr int kWaves = 16;

// 16 TT tokens per work group; wave = (tile p, slice ks) of PT = kWaves / KS tiles of 16
// weight rows (gated: 16 gate and 16 up rows); slice ks takes the blocks b = ks, ks + KS, ...
// and the slices' sums meet in LDS in order.
template <int TT, int KS, bool GATED>
__global__ __launch_bounds__(kWaves * 64) void product_split_kernel(const ProductArgs a) {
    constexpr int PT = kWaves / KS, M = GATED ? 2 : 1;
    static_assert(!GATED || PT == 8, "a gated work group covers one 128-column output group");
    __shared__ f32x4 red[KS > 1 ? KS - 1 : 1][PT][M][TT][64];
    __shared__ uint32_t amax[GATED ? 8 : 1][TT * 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int p = wave % PT, ks = wave / PT;
    const int N = a.N, K = a.K, KB = (K + kBlock - 1) / kBlock, NB = (N + kBlock - 1) / kBlock;
    const RowSpan s = span_of<16 * TT>(a, blockIdx.y);
    if (s.n == 0) return;
    const int n0 = (blockIdx.x * PT + p) * 16;  // first weight row of the wave's tile
    const uint8_t* wrow[M];
    const float* ws[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const size_t mat = (size_t)s.e * M + m;
        const int row = min(n0 + c, N - 1);  // clamped, valid
        wrow[m] = a.w + (mat * N + row) * (size_t)K;
        ws[m] = a.w_scale + (mat * NB + min(n0, N - 1) / kBlock) * (size_t)KB;
    }
    const uint8_t* xrow[TT];
    const float* xs[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const size_t row = s.row0 + min(16 * t + c, s.n - 1);  // clamped, valid
        xrow[t] = a.x + row * (size_t)K;
        xs[t] = a.x_scale + row * (size_t)KB;
    }
    f32x4 acc[M][TT];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (n0 < N) {
        for (int b = ks; b < KB; b += KS) {
            const int k0 = b * kBlock + 32 * g;
            const bool live = k0 < K;       // K is a multiple of 64: the last block may be half
            const int kk = live ? k0 : 0;   // clamped, valid
            const u32x4 zero = {0u, 0u, 0u, 0u};
            Operand w[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const u32x4 lo = *(const u32x4*)(wrow[m] + kk), hi = *(const u32x4*)(wrow[m] + kk + 16);
                w[m] = operand(live ? lo : zero, live ? hi : zero);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const u32x4 lo = *(const u32x4*)(xrow[t] + kk), hi = *(const u32x4*)(xrow[t] + kk + 16);
                const Operand x = operand(live ? lo : zero, live ? hi : zero);
                const float xsc = xs[t][b];
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const f32x4 d = block_product(w[m], x);
                    const float f = xsc * ws[m][b];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][t][i] = __builtin_fmaf(d[i], f, acc[m][t][i]);
                }
            }
        }
    }
    if constexpr (KS > 1) {
        if (ks > 0) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int t = 0; t < TT; ++t) red[ks - 1][p][m][t][lane] = acc[m][t];
        }
        __syncthreads();
        if (ks == 0) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    for (int j = 0; j < KS - 1; ++j) acc[m][t] += red[j][p][m][t][lane];
        }
    }
    const int o = n0 + 4 * g;
    if constexpr (!GATED) {
        if (ks > 0) return;
#pragma unroll
        for (int t = 0; t < TT; ++t)
            if (16 * t + c < s.n) store4(a, (size_t)s.row0 + 16 * t + c, o, acc[0][t]);
    } else {
        float h[TT][4];
        if (ks == 0) {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[t][i] = silu(acc[0][t][i]) * acc[1][t][i];
                    if (n0 < N) m = max_magnitude(m, h[t][i]);
                }
                m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
                if (g == 0) amax[p][16 * t + c] = m;
            }
        }
        __syncthreads();
        if (ks > 0 || n0 >= N) return;
        const int groups = (N + kBlock - 1) / kBlock;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, amax[j][16 * t + c]);
            float scale;
            uint32_t codes[1];
            e4m3_codes<4>(h[t], __uint_as_float(m), &scale, codes);
            if (16 * t + c >= s.n) continue;
            const size_t row = (size_t)s.row0 + 16 * t + c;
            *(uint32_t*)((uint8_t*)a.y + row * (size_t)N + o) = codes[0];
            if (p == 0 && g == 0) a.y_scale[row * (size_t)groups + n0 / kBlock] = scale;
        }
    }
}

template <int TT, int KS, bool GATED>
void launch_split(const ProductArgs& a, int tiles, hipStream_t s) {
    constexpr int PT = kWaves / KS;
    const dim3 grid((a.N + 16 * PT - 1) / (16 * PT), tiles);
    product_split_kernel<TT, KS, GATED><<<grid, kWaves * 64, 0, s>>>(a);
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
    const int tiles = a.map ? a.map_bound : (a.rows + 31) / 32;
    if (a.gated) launch_split<2, 2, true>(a, tiles, s);
    else launch_split<2, 4, false>(a, tiles, s);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
