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
// K is a multiple of 64: a last block of 64 columns takes the place of both halves, in W and
// in x, and its factor is halved.  That doubles every term exactly, and asks for no zeros in the
// place of the missing columns.
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
        if (j >= min(*a.n_map, a.map_bound)) return s;
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
            const int kk = k0 < K ? k0 : k0 - 64;
            const float part = b == KB - 1 && (K & 64) ? 0.5f : 1.0f;
            Operand w[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const u32x4 lo = *(const u32x4*)(wrow[m] + kk), hi = *(const u32x4*)(wrow[m] + kk + 16);
                w[m] = operand(lo, hi);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const u32x4 lo = *(const u32x4*)(xrow[t] + kk), hi = *(const u32x4*)(xrow[t] + kk + 16);
                const Operand x = operand(lo, hi);
                const float xsc = xs[t][b] * part;
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

// ---------------------------------------------------------------------------
// Tiles: BM tokens by BN weight rows per work group of 8 waves, WM x WN of them; x and W go
// through LDS in S stages of one block of 128 columns each, loaded straight into it.
//
// LDS holds a row of a stage as eight 16-byte pieces, piece c at place c ^ (row & 7): the
// loads write LDS in lane order, so a lane fetches the piece that belongs at its place, and
// sixteen lanes that read the same piece of sixteen rows meet all banks.
// ---------------------------------------------------------------------------
constexpr int kTileThreads = 512;
constexpr int kMaxBlocks = MOE_MAX_D / kBlock;

// Loads of 16 (4) bytes per lane straight into LDS at lds + 16 (4) * lane, from the buffer rsrc
// at voff + soff; lds, rsrc and soff are the wave's.  Written out because the compiler waits
// for all of its own such loads before any read of the same LDS object, also of another stage;
// here a stage's loads are waited for by count, before the barrier that hands the stage out.
// They have no result registers.  M0 takes the LDS address (one wait state before its use); no
// other instruction of these kernels reads it.
__device__ __forceinline__ void load16_lds(const u32x4& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %0, %2 offen lds"
                 ::"s"(rsrc), "v"(voff), "s"(soff), "s"(lds) : "memory");
#endif
}
__device__ __forceinline__ void load4_lds(const u32x4& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %1, %0, %2 offen lds"
                 ::"s"(rsrc), "v"(voff), "s"(soff), "s"(lds) : "memory");
#endif
}

// The buffer of everything from p on (p the same in the whole wave).
__device__ __forceinline__ u32x4 buffer_from(const void* p) {
    const uint64_t u = (uint64_t)p;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(u >> 32) & 0xFFFFu)), 0xFFFFFFFFu,
                 0x00020000u};
}

// s_waitcnt vmcnt(N), leaving the other counters alone (vmcnt in bits 3:0 and 15:14, expcnt
// 6:4, lgkmcnt 11:8).
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Tile id of this work group: work groups go to the 8 XCDs in turn, so consecutive ids of
// one XCD are made neighbouring tiles (of which the XCD's L2 holds what they share).
__device__ __forceinline__ int neighbour_id(int id, int total) {
    const int per = total >> 3, rest = total & 7, xcd = id & 7, at = id >> 3;
    return xcd * per + min(xcd, rest) + at;
}

template <bool E4M3>
struct TileOperand {
    using type = Operand;
};
typedef int i32x8 __attribute__((ext_vector_type(8)));
template <>
struct TileOperand<true> {
    using type = i32x8;
};

// E4M3: the matrix cores' own 8-bit products (see the top), for bf16 outputs.
template <int BM, int BN, int WM, int WN, int S, bool E4M3, bool GATED, bool MAPPED, bool ROTATE>
__global__ __launch_bounds__(kTileThreads) void product_tile_kernel(const ProductArgs a) {
    static_assert(WM * WN == 8 && S >= 2 && S <= 4 && (!GATED || BN == 256), "shape");
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16, M = GATED ? 2 : 1;
    constexpr int kX = BN * kBlock, kXs = kX + BM * kBlock;
    constexpr int kScales = BM < 64 ? 256 : 4 * BM, kStage = kXs + kScales;  // (a load writes 256 bytes)
    constexpr int kWLoads = BN / 64, kXLoads = (BM + 63) / 64, kLoads = kWLoads + kXLoads + 1;
    __shared__ __attribute__((aligned(16))) unsigned char lds[S * kStage];
    __shared__ float s_ws[2][kMaxBlocks];  // the scales of W's two halves (gated: gate, up)
    __shared__ uint32_t amax[GATED ? WN : 1][GATED ? BM : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
    const int N = a.N, K = a.K, KB = (K + kBlock - 1) / kBlock, NB = (N + kBlock - 1) / kBlock;
    constexpr int kCols = BN / M;  // output columns of a tile
    const int n_tiles = (N + kCols - 1) / kCols;

    RowSpan s;
    int nt;
    if constexpr (MAPPED) {  // neighbours: the columns of one tile of rows
        const int total = min(*a.n_map, a.map_bound) * n_tiles;
        if ((int)blockIdx.x >= total) return;
        const int id = neighbour_id(blockIdx.x, total);
        nt = id % n_tiles;
        s = span_of<BM>(a, id / n_tiles);
    } else {  // neighbours: 8 tiles of rows by a few of columns
        const int m_tiles = (a.rows + BM - 1) / BM, id = neighbour_id(blockIdx.x, m_tiles * n_tiles);
        const int group = id / (8 * n_tiles), in = id - group * 8 * n_tiles;
        const int high = min(8, m_tiles - 8 * group);
        nt = in / high;
        s = span_of<BM>(a, 8 * group + in % high);
    }
    if (s.n == 0) return;
    const int n0 = nt * kCols;

    // this lane's piece of every load: row lane / 8 of 8, place lane % 8
    const int piece = (lane & 7) ^ (lane >> 3);
    const uint8_t* wbase = a.w + ((size_t)s.e * M * N + n0) * (size_t)K;
    const uint8_t* xbase = a.x + (size_t)s.row0 * K;
    uint32_t woff[kWLoads], xoff[kXLoads];
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
        const int r = 8 * (wave + 8 * j) + (lane >> 3);
        if (GATED) {
            woff[j] = (uint32_t)min(r & 127, N - 1 - n0) * (uint32_t)K + 16 * piece;
        } else {
            woff[j] = (uint32_t)min(r, N - 1 - n0) * (uint32_t)K + 16 * piece;
        }
    }
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) {
        const int r = (8 * (wave + 8 * j) + (lane >> 3)) % BM;
        xoff[j] = (uint32_t)min(r, s.n - 1) * (uint32_t)K + 16 * piece;
    }
    const uint32_t soff = (uint32_t)(s.row0 + min((64 * wave + lane) % BM, s.n - 1)) * (uint32_t)KB * 4u;
    const u32x4 w_rsrc = buffer_from(wbase), x_rsrc = buffer_from(xbase), s_rsrc = buffer_from(a.x_scale);
    const u32x4 up_rsrc = buffer_from(wbase + (GATED ? (size_t)N * K : 0));
    const bool half = K & 64;  // the last block has 64 columns
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;

    // Block b of the tile into the stage at `at` (the second half of a half block is its first
    // again).
    auto load = [&](uint32_t at, int b) {
        const uint32_t back = half && b == KB - 1 && piece >= 4 ? 64u : 0u;
        const uint32_t to = lds0 + at + 1024u * (uint32_t)wave;
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            load16_lds(GATED && j >= kWLoads / 2 ? up_rsrc : w_rsrc, woff[j] - back, b * kBlock, to + 8192u * j);
#pragma unroll
        for (int j = 0; j < kXLoads; ++j)
            load16_lds(x_rsrc, xoff[j] - back, b * kBlock,
                       lds0 + at + kX + (1024u * (uint32_t)(wave + 8 * j)) % (uint32_t)(BM * kBlock));
        load4_lds(s_rsrc, soff, 4 * b, lds0 + at + kXs + (256u * (uint32_t)wave) % (uint32_t)kScales);
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // row of W in the stage of this wave's tile i, and its half
    auto w_row = [&](int i) {
        if (!GATED) return (wn * NT + i) * 16;
        return (i < NT / 2 ? 0 : 128) + (wn * (NT / 2) + i % (NT / 2)) * 16;
    };
    auto compute = [&](uint32_t at, int b) {
        const unsigned char* buf = lds + at;
        const int lo = ((2 * g) ^ (c & 7)) << 4, hi = ((2 * g + 1) ^ (c & 7)) << 4;
        typename TileOperand<E4M3>::type w[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const unsigned char* p = buf + (w_row(i) + c) * kBlock;
            const u32x4 u = *(const u32x4*)(p + lo), v = *(const u32x4*)(p + hi);
            if constexpr (E4M3) w[i] = i32x8{(int)u[0], (int)u[1], (int)u[2], (int)u[3], (int)v[0], (int)v[1], (int)v[2], (int)v[3]};
            else w[i] = operand(u, v);
        }
        float ws[M];
        ws[0] = s_ws[!GATED && wn * NT * 16 >= 128 ? 1 : 0][b];
        if constexpr (GATED) ws[1] = s_ws[1][b];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int r = wm * MT * 16 + 16 * t;
            if (MAPPED && r >= s.n) break;  // (the same for the whole wave)
            const unsigned char* p = buf + kX + (r + c) * kBlock;
            const u32x4 u = *(const u32x4*)(p + lo), v = *(const u32x4*)(p + hi);
            const float xs = *(const float*)(buf + kXs + 4 * (r + c));
            float f[M];
#pragma unroll
            for (int m = 0; m < M; ++m) f[m] = xs * ws[m];
            if constexpr (E4M3) {
                const i32x8 x = {(int)u[0], (int)u[1], (int)u[2], (int)u[3], (int)v[0], (int)v[1], (int)v[2], (int)v[3]};
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    // formats 0 (e4m3); scales 0 select the instruction without block exponents
                    const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        w[i], x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[t][i][q] = __builtin_fmaf(d[q], f[GATED && i >= NT / 2 ? M - 1 : 0], acc[t][i][q]);
                }
            } else {
                const Operand x = operand(u, v);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const f32x4 d = block_product(w[i], x);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[t][i][q] = __builtin_fmaf(d[q], f[GATED && i >= NT / 2 ? M - 1 : 0], acc[t][i][q]);
                }
            }
        }
    };
    // Every tile begins with another block of columns: W's rows lie a power of two apart, and
    // tiles in step would read the same few memory channels.
    const int turn = ROTATE ? (nt + s.e) % KB : 0;
    auto block = [&](int i) { return ROTATE ? (i + turn < KB ? i + turn : i + turn - KB) : i; };
#pragma unroll
    for (int j = 0; j < S - 1; ++j)
        if (j < KB) load(j * kStage, block(j));
    {
        const int h = tid >> 6;
        if (h < 2 && lane < KB) {
            const int nb = GATED ? n0 / kBlock : min(n0 / kBlock + h * (BN > 128 ? 1 : 0), NB - 1);
            const float ws = a.w_scale[(((size_t)s.e * M + (GATED ? h : 0)) * NB + nb) * (size_t)KB + lane];
            s_ws[h][lane] = half && lane == KB - 1 ? 0.5f * ws : ws;
        }
    }
    // Step i: wait for its block's loads (those of the next S - 2 blocks stay in flight), start
    // those of block i + S - 1 into the stage that every wave has left, multiply.
    uint32_t here = 0;
    for (int i = 0; i < KB; ++i) {
        if (S > 3 && i + 2 < KB) wait_loads<(S > 3 ? 2 * kLoads : 0)>();
        else if (S > 2 && i + 1 < KB) wait_loads<(S > 2 ? kLoads : 0)>();
        else wait_loads<0>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (s_ws, once)
        __builtin_amdgcn_s_barrier();
        const uint32_t free_at = here == 0 ? (S - 1) * kStage : here - kStage;
        if (i + S - 1 < KB) load(free_at, block(i + S - 1));
        compute(here, block(i));
        here = here == (S - 1) * kStage ? 0 : here + kStage;
    }

    if constexpr (!GATED) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int r = wm * MT * 16 + 16 * t + c;
            if (r >= s.n) continue;
#pragma unroll
            for (int i = 0; i < NT; ++i) store4(a, (size_t)s.row0 + r, n0 + w_row(i) + 4 * g, acc[t][i]);
        }
    } else {
        constexpr int H = NT / 2;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const bool live = n0 + w_row(i) < N;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[t][i][q] = silu(acc[t][i][q]) * acc[t][i + H][q];
                    if (live) m = max_magnitude(m, acc[t][i][q]);
                }
            }
            m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
            if (g == 0) amax[wn][wm * MT * 16 + 16 * t + c] = m;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int r = wm * MT * 16 + 16 * t + c;
            if (r >= s.n) continue;
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < WN; ++j) m = max(m, amax[j][r]);
            const size_t row = (size_t)s.row0 + r;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int o = n0 + w_row(i) + 4 * g;
                float h[4] = {acc[t][i][0], acc[t][i][1], acc[t][i][2], acc[t][i][3]}, scale;
                uint32_t codes[1];
                e4m3_codes<4>(h, __uint_as_float(m), &scale, codes);
                if (o < N) *(uint32_t*)((uint8_t*)a.y + row * (size_t)N + o) = codes[0];
                if (i == 0 && wn == 0 && g == 0) a.y_scale[row * (size_t)NB + nt] = scale;
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, int S, bool E4M3, bool GATED, bool MAPPED, bool ROTATE>
void launch_tile(const ProductArgs& a, int tiles, hipStream_t s) {
    constexpr int kCols = GATED ? BN / 2 : BN;
    const unsigned grid = (unsigned)tiles * (unsigned)((a.N + kCols - 1) / kCols);
    product_tile_kernel<BM, BN, WM, WN, S, E4M3, GATED, MAPPED, ROTATE><<<grid, kTileThreads, 0, s>>>(a);
}

// Rows of a tile map of BM-row tiles (dense: the rows themselves).
template <int BM>
int tiles_of(ProductArgs& a) {
    if (!a.map) return (a.rows + BM - 1) / BM;
    if (BM == 128) {
        a.map = a.map128;
        a.n_map = a.n_map128;
        a.map_bound = a.map128_bound;
    }
    return a.map_bound;
}

}  // namespace

hipError_t launch_product(const ProductArgs& a0, hipStream_t s) {
    ProductArgs a = a0;
    const int per = a.map ? (a.rows + a.E - 1) / a.E : a.rows;  // rows that share a matrix
    const long long wgs256 = (long long)((a.N + 255) / 256) * (a.map ? min(a.rows, a.E) : (a.rows + 31) / 32);
    if (a.map) {
        if (per <= 16) {
            const int tiles = tiles_of<32>(a);
            if (a.gated) launch_tile<32, 256, 1, 8, 4, false, true, true, true>(a, tiles, s);
            else if (wgs256 >= 128) launch_tile<32, 256, 1, 8, 4, false, false, true, true>(a, tiles, s);
            else launch_split<2, 4, false>(a, tiles, s);
        } else if (a.gated) {
            launch_tile<128, 256, 2, 4, 3, false, true, true, true>(a, tiles_of<128>(a), s);
        } else {
            launch_tile<128, 256, 2, 4, 3, false, false, true, true>(a, tiles_of<128>(a), s);
        }
    } else if (per <= 16) {
        const int tiles = tiles_of<32>(a);
        if (a.gated) launch_split<1, 2, true>(a, tiles_of<16>(a), s);
        else if (wgs256 >= 128) launch_tile<32, 256, 1, 8, 4, false, false, false, true>(a, tiles, s);
        else if (a.N < 4096) launch_split<1, 16, false>(a, tiles_of<16>(a), s);
        else launch_split<1, 8, false>(a, tiles_of<16>(a), s);
    } else if (a.gated) {
        if (a.rows >= 2048) launch_tile<256, 256, 2, 4, 2, false, true, false, false>(a, tiles_of<256>(a), s);
        else if (a.rows <= 64) launch_tile<64, 256, 2, 4, 3, false, true, false, true>(a, tiles_of<64>(a), s);
        else launch_tile<128, 256, 2, 4, 3, false, true, false, false>(a, tiles_of<128>(a), s);
    } else {
        const bool wide = (long long)((a.N + 255) / 256) * ((a.rows + 255) / 256) >= 256;
        if (wide) {
            if (a.out_bf16) launch_tile<256, 256, 2, 4, 2, true, false, false, false>(a, tiles_of<256>(a), s);
            else launch_tile<256, 256, 2, 4, 2, false, false, false, false>(a, tiles_of<256>(a), s);
        } else if (a.rows <= 64) {
            launch_tile<64, 128, 2, 4, 3, false, false, false, true>(a, tiles_of<64>(a), s);
        } else {
            launch_tile<128, 128, 2, 4, 3, false, false, false, false>(a, tiles_of<128>(a), s);
        }
    }
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
