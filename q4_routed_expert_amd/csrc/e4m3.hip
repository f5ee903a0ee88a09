// e4m3.hip -- products of e4m3 rows with e4m3 matrices, one scale per token and 128
// columns of x and one per 128 x 128 block of W (moe_linear_scaled, moe_experts_scaled):
//
//   y[t][n] = sum over blocks b of xs[t][b] ws[n / 128][b] sum over k in b of x[t][k] w[n][k]
//
// Codes become bf16 on the way into the matrix cores (exactly: 4 significant bits, exponents
// -9 .. 8), four v_mfma_f32_16x16x32_bf16 per block with 16 weight rows as A and 16 tokens
// as B; then the block's fp32 sum is scaled and added by four fused multiply-adds.  The matrix
// cores' own e4m3 products are twice as fast (3670 instead of 1830 TFLOP/s, nothing else
// running), but they cut every product at 13 bits below the largest among eight columns: sums
// of 128 normally distributed values came out 1.5e-5 off (2-norm), through bf16 9e-9.  In usual sums
// that is far below the rounding of a bf16 output (2e-3), but where large products cancel, small
// ones next to them are lost.  So bf16 outputs take them from 128 rows (of an expert, on average)
// on, where a product is bound by the matrix cores: 2 rows operations a byte of W at 1227 TFLOP/s
// and 5.1 TB/s meet at 120.  fp32 outputs and the scales of gated ones would show them always.
// A block's sum is the same in any order of its columns, as long as A and B hold the same
// ones: lane (r = lane & 15, g = lane >> 4) holds columns 32 g .. + 31 of row r of both.  In D
// lane (c, g) holds token c, weight rows 4 g .. + 3, so a lane's factor xs * ws is one number
// per 16 tokens and block.
//
// K is a multiple of 64: a last block of 64 columns takes the place of both halves, in W and
// in x, and its factor is halved.  That doubles every term exactly, and asks for no zeros in the
// place of the missing columns.
//
// Gated output: the matrix holds gate and up rows; a wave computes the same rows of each, so
// both sums of a column are in one lane, and silu(gate) * up leaves in e4m3.
//
// Bounds and times (three states in turn): 8192^3 in bf16 560 us, 1.96 PFLOP/s (matrix cores
// and the LDS reads that feed them: multiplying alone 424 us, loading alone 404); in fp32 970 us,
// 1.13 PFLOP/s (vector ALUs: a conversion for two codes, a multiply-add for an output and block,
// and a matrix instruction holds their issue for as long as three of them).  Expert products
// stream weights: 8 tokens through 256 experts of 2 x 512 rows, K = 2048, 24 us (5.0 TB/s); 2048
// tokens 155 us (130 of multiplying alone, 113 of loading alone); 4096 tokens through 2048
// rows, K = 512, in bf16 96 us (4.4 TB/s).  One token, 2048 x 2048: 3.7 us.
#include "e4m3.h"
#include "ops.h"

namespace q4moe {
namespace {

// What a work group's rows are: rows row0 .. row0 + n - 1 of x and y, matrix e.
struct RowSpan {
    int row0, n, e;
};

// The maps are read through scalar loads: nothing writes them while a kernel runs, and a vector
// load would be waited for behind every load of a tile that is in flight.
typedef const __attribute__((address_space(4))) int32_t* ScalarInts;
__device__ __forceinline__ int scalar_int(const int32_t* p, size_t i) { return ((ScalarInts)(uintptr_t)p)[i]; }

// Tile j of TR rows: of the rows themselves, or of the map of expert-sorted rows.  Map
// entries come from device memory: rows out of range are no tile, experts are brought into it.
template <int TR>
__device__ __forceinline__ RowSpan span_of(const ProductArgs& a, int j) {
    RowSpan s{0, 0, 0};
    if (!a.map) {
        s.row0 = j * TR;
        s.n = a.rows - s.row0;
    } else {
        const int row = scalar_int(a.map, 2 * (size_t)j + 1);
        if (row < 0 || row >= a.rows) return s;
        s.e = min(max(scalar_int(a.map, 2 * (size_t)j), 0), a.E - 1);
        s.row0 = row;
        s.n = min(scalar_int(a.offsets, s.e + 1), a.rows) - row;
    }
    s.n = min(max(s.n, 0), TR);
    return s;
}

// Tiles of the map that are there.
__device__ __forceinline__ int mapped_tiles(const ProductArgs& a) {
    return min(scalar_int(a.n_map, 0), a.map_bound);
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

// Sixteen or eight bytes at a 2-byte address (one store: the hardware takes any alignment, and
// rows of an odd number of columns begin anywhere).
template <int N>
struct __attribute__((packed, aligned(2))) Words {
    uint32_t w[N];
};

// Four sums of one token, weight rows o .. o + 3.
__device__ __forceinline__ void store4(const ProductArgs& a, size_t row, int o, const f32x4& v) {
    const size_t at = row * (size_t)a.N + o;
    if (o + 4 <= a.N) {
        if (a.out_bf16) *(Words<2>*)((uint16_t*)a.y + at) = Words<2>{{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}};
        else *(Words<4>*)((float*)a.y + at) = __builtin_bit_cast(Words<4>, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (o + i >= a.N) break;
        if (a.out_bf16) ((uint16_t*)a.y)[at + i] = f32_to_bf16(v[i]);
        else ((float*)a.y)[at + i] = v[i];
    }
}

// Eight sums of one token in bf16, weight rows o .. o + 7.
__device__ __forceinline__ void store8(const ProductArgs& a, size_t row, int o, const Words<4>& v) {
    uint16_t* at = (uint16_t*)a.y + row * (size_t)a.N + o;
    if (o + 8 <= a.N) {
        *(Words<4>*)at = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (o + i < a.N) at[i] = (uint16_t)(v.w[i / 2] >> (16 * (i & 1)));
}

// ---------------------------------------------------------------------------
// Few tokens and few weight rows: 16 weight rows and 16 TT tokens per work group, whose 16
// waves share the blocks of columns (wave w takes w, w + 16, ...) and whose sums meet in LDS in
// wave order.  Operands come straight from memory: with one wave a block there is one round
// trip.
// ---------------------------------------------------------------------------
constexpr int kWaves = 16;

template <int TT>
__global__ __launch_bounds__(kWaves * 64) void product_split_kernel(const ProductArgs a) {
    __shared__ f32x4 red[kWaves][TT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int N = a.N, K = a.K, KB = (K + kBlock - 1) / kBlock;
    const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16 * TT;
    const uint8_t* wrow = a.w + (size_t)min(n0 + c, N - 1) * K;  // (clamped rows are not stored)
    const float* ws = a.w_scale + (size_t)(n0 / kBlock) * KB;
    const uint8_t* xrow[TT];
    const float* xs[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const size_t row = min(t0 + 16 * t + c, a.rows - 1);
        xrow[t] = a.x + row * (size_t)K;
        xs[t] = a.x_scale + row * (size_t)KB;
    }
    f32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = wave; b < KB; b += kWaves) {
        const int k0 = b * kBlock + 32 * g;
        const int kk = k0 < K ? k0 : k0 - 64;
        const float f = ws[b] * (b == KB - 1 && (K & 64) ? 0.5f : 1.0f);
        const Operand w = operand(*(const u32x4*)(wrow + kk), *(const u32x4*)(wrow + kk + 16));
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const Operand x = operand(*(const u32x4*)(xrow[t] + kk), *(const u32x4*)(xrow[t] + kk + 16));
            const float ft = xs[t][b] * f;
            f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[j], x.v[j], d, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(d[i], ft, acc[t][i]);
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) red[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave >= TT) return;
    f32x4 sum = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += red[w][wave][lane];
    const int row = t0 + 16 * wave + c;
    if (row < a.rows) store4(a, row, n0 + 4 * g, sum);
}

template <int TT>
void launch_split(const ProductArgs& a, hipStream_t s) {
    const dim3 grid((a.N + 15) / 16, (a.rows + 16 * TT - 1) / (16 * TT));
    product_split_kernel<TT><<<grid, kWaves * 64, 0, s>>>(a);
}

// ---------------------------------------------------------------------------
// Tiles: BM tokens by BN weight rows per work group of WM x WN waves; x and W go
// through LDS in S stages of one block of 128 columns each, loaded straight into it.
//
// One work group per CU (or two or three, where their LDS fits) walks its share of the tiles,
// and its stages run on from one tile to the next: the loads of the next tile are under way
// while the last blocks of this one are multiplied and its outputs are stored.  (A work group
// for every tile: the down products of 4096 tokens 159 instead of 147 us, 8192^3 the same.)
//
// What was tried and is slower: halves of the waves that take turns at reading and at
// multiplying (8192^3 837 us: loads and the other half's LDS reads meet), sixteen waves
// (expert products + 5 %), touching blocks ahead of their loads so that L2 has them (8192^3 + 6 %).
//
// LDS holds a row of a stage as eight 16-byte pieces, piece p at place p ^ (row & 7): the
// loads write LDS in lane order, so a lane fetches the piece that belongs at its place.  A lane
// of group g multiplies pieces g and g + 4 (with 2 g and 2 g + 1, half of the reads met in a bank).
// ---------------------------------------------------------------------------
constexpr int kCus = 256;

template <int N>
struct Int {
    static constexpr int value = N;
};

// Loads of 16 (4) bytes per lane straight into LDS at lds + 16 (4) * lane, from the buffer rsrc
// at voff + soff; lds, rsrc and soff are the wave's.  Written out because the compiler waits
// for all of its own such loads before any read of the same LDS object, also of another stage;
// here a stage's loads are waited for by count, before the barrier that hands the stage out.
// They have no result registers.  M0 takes the LDS address (one wait state before its use); no
// other instruction of these kernels reads it.
// NT: not kept in the caches for others.
template <bool NT = false>
__device__ __forceinline__ void load16_lds(const u32x4& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %0, %2 offen nt lds"
                     ::"s"(rsrc), "v"(voff), "s"(soff), "s"(lds) : "memory");
    else
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

// s_waitcnt vmcnt(N) lgkmcnt(0), before a barrier: all but the newest N loads are there, and this
// wave's reads of LDS are done, so that others may write what it read (vmcnt in bits 3:0 and
// 15:14, expcnt 6:4, lgkmcnt 11:8).
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4));
}

typedef int i32x8 __attribute__((ext_vector_type(8)));
template <bool E4M3>
struct TileOperand {
    using type = Operand;
};
template <>
struct TileOperand<true> {
    using type = i32x8;
};

template <bool E4M3>
__device__ __forceinline__ typename TileOperand<E4M3>::type tile_operand(const u32x4& u, const u32x4& v) {
    if constexpr (E4M3) return i32x8{(int)u[0], (int)u[1], (int)u[2], (int)u[3], (int)v[0], (int)v[1], (int)v[2], (int)v[3]};
    else return operand(u, v);
}

// A block's products of NT tiles of weight rows with one of tokens; four independent chains
// take turns, so that no product waits for the one before.
template <int NT>
__device__ __forceinline__ void tile_products(f32x4 (&d)[NT], const Operand (&w)[NT], const Operand& x) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i)
            d[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                w[i].v[j], x.v[j], j == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : d[i], 0, 0, 0);
}

template <int NT>
__device__ __forceinline__ void tile_products(f32x4 (&d)[NT], const i32x8 (&w)[NT], const i32x8& x) {
    // formats 0 (e4m3) for both; scales 0 select the instruction without block exponents
#pragma unroll
    for (int i = 0; i < NT; ++i)
        d[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[i], x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// E4M3: the matrix cores' own 8-bit products (see the top).
template <int BM, int BN, int WM, int WN, int S, bool E4M3, bool GATED, bool MAPPED>
__global__ __launch_bounds__(WM * WN * 64) void product_tile_kernel(const ProductArgs a) {
    constexpr int kW = WM * WN;
    static_assert((kW == 8 || kW == 4) && BM <= 32 * kW && S >= 2 && S <= 4 && (!GATED || BN == 256) && (!MAPPED || BM / WM <= 64), "shape");
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16, M = GATED ? 2 : 1;
    // a stage: W's rows, x's rows, x's scales (a load writes 256 bytes), the two scales of W
    constexpr int kX = BN * kBlock, kXs = kX + BM * kBlock, kWs = kXs + (BM < 64 ? 256 : 4 * BM), kStage = kWs + 256;
    constexpr int kWLoads = BN / (8 * kW), kXLoads = (BM + 8 * kW - 1) / (8 * kW), kLoads = kWLoads + kXLoads + 1;
    __shared__ __attribute__((aligned(16))) unsigned char lds[S * kStage];
    __shared__ uint32_t amax[GATED ? WN : 1][GATED ? BM : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
    const int N = a.N, K = a.K, KB = (K + kBlock - 1) / kBlock, NB = (N + kBlock - 1) / kBlock;
    constexpr int kCols = BN / M;  // output columns of a tile
    const int n_tiles = (N + kCols - 1) / kCols;
    const int m_tiles = MAPPED ? mapped_tiles(a) : (a.rows + BM - 1) / BM;

    // Work groups go to the 8 XCDs in turn: an XCD takes a run of neighbouring tiles, its work
    // groups the next ones of it in turn, so that its L2 holds what they share.
    const int total = m_tiles * n_tiles, xcd = blockIdx.x & 7, per_xcd = gridDim.x >> 3;
    const int end = (int)((long long)total * (xcd + 1) >> 3);
    const int first = (int)((long long)total * xcd >> 3) + ((int)blockIdx.x >> 3);
    if (first >= end) return;

    // Tile `id`: its rows and its column tile.  Neighbours are, of expert-sorted rows, the
    // columns of one tile of rows; else 8 tiles of rows by a few of columns.
    auto tile = [&](int id, int* nt) {
        if constexpr (MAPPED) {
            *nt = id % n_tiles;
            return span_of<BM>(a, id / n_tiles);
        } else {
            const int group = id / (8 * n_tiles), in = id - group * 8 * n_tiles;
            const int high = min(8, m_tiles - 8 * group);
            *nt = in / high;
            return span_of<BM>(a, 8 * group + in % high);
        }
    };

    // Loading: tile l_id, block l_b; this lane's piece of every load is row lane / 8 of 8,
    // place lane % 8.
    const int piece = (lane & 7) ^ (lane >> 3);
    const bool half = K & 64;  // the last block has 64 columns
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    int l_id = first, l_b = 0;
    uint32_t woff[kWLoads], xoff[kXLoads], soff;
    u32x4 w_rsrc, up_rsrc, x_rsrc, s_rsrc;
    auto enter = [&](int id) {
        int nt;
        const RowSpan s = tile(id, &nt);
        const int n0 = nt * kCols, last = max(s.n, 1) - 1;
        const uint8_t* w = a.w + ((size_t)s.e * M * N + n0) * (size_t)K;
        w_rsrc = buffer_from(w);
        up_rsrc = buffer_from(w + (GATED ? (size_t)N * K : 0));
        x_rsrc = buffer_from(a.x + (size_t)s.row0 * K);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j) {
            const int r = 8 * (wave + kW * j) + (lane >> 3);
            woff[j] = (uint32_t)min(GATED ? r & 127 : r, N - 1 - n0) * (uint32_t)K + 16 * piece;
        }
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) {
            const int r = (8 * (wave + kW * j) + (lane >> 3)) % BM;
            xoff[j] = (uint32_t)min(r, last) * (uint32_t)K + 16 * piece;
        }
        // half of the waves fetch x's scales, the others W's: of its two halves, or of gate and up
        if (wave < kW / 2) {
            s_rsrc = buffer_from(a.x_scale + (size_t)s.row0 * KB);
            soff = 4u * (uint32_t)min((64 * wave + lane) % BM, last) * (uint32_t)KB;
        } else {
            const int nb = n0 / kBlock, other = GATED ? NB : BN > 128 ? min(nb + 1, NB - 1) - nb : 0;
            s_rsrc = buffer_from(a.w_scale + ((size_t)s.e * M * NB + nb) * (size_t)KB);
            soff = 4u * (uint32_t)((lane & 1) * other) * (uint32_t)KB;
        }
    };
    // The next block, if there is one, into the stage at `at` (the second half of a half block
    // is its first again).
    auto load = [&](uint32_t at) {
        if (l_id >= end) return;
        const uint32_t back = half && l_b == KB - 1 && piece >= 4 ? 64u : 0u;
        const uint32_t to = lds0 + at + 1024u * (uint32_t)wave;
        auto load_w = [&](auto nt) {
#pragma unroll
            for (int j = 0; j < kWLoads; ++j)
                load16_lds<decltype(nt)::value != 0>(GATED && j >= kWLoads / 2 ? up_rsrc : w_rsrc, woff[j] - back,
                                                     l_b * kBlock, to + 1024u * kW * j);
        };
        if ((BM == 32 || MAPPED) && BN == 256 && a.stream) load_w(Int<1>{});
        else load_w(Int<0>{});
#pragma unroll
        for (int j = 0; j < kXLoads; ++j)
            load16_lds(x_rsrc, xoff[j] - back, l_b * kBlock,
                       lds0 + at + kX + (1024u * (uint32_t)(wave + kW * j)) % (uint32_t)(BM * kBlock));
        load4_lds(s_rsrc, soff, 4 * l_b,
                  lds0 + at + (wave < kW / 2 ? kXs + (256u * (uint32_t)wave) % (uint32_t)(kWs - kXs) : (uint32_t)kWs));
        if (++l_b == KB) {
            l_b = 0;
            l_id += per_xcd;
            if (l_id < end) enter(l_id);
        }
    };

    // row of W in a stage of this wave's tile i
    auto w_row = [&](int i) {
        if (!GATED) return (wn * NT + i) * 16;
        return (i < NT / 2 ? 0 : 128) + (wn * (NT / 2) + i % (NT / 2)) * 16;
    };
    // first row of this wave's 16 tokens t (few rows are shared evenly)
    auto x_row = [&](int t) { return MAPPED ? 16 * (t * WM + wm) : 16 * (wm * MT + t); };
    f32x4 acc[MT][NT];
    // The block in the stage at `at`, for the first TL of this wave's 16-token tiles.  The
    // operands of 16 tokens are read while those of the 16 before are multiplied, whose sums, of
    // bf16 products, are added one turn later still (of 8-bit ones at once: with two tiles' sums
    // in registers the largest tile spills, 8192^3 633 instead of 567 us).
    auto compute = [&](auto live, uint32_t at, float part) {
        constexpr int TL = decltype(live)::value;
        using Op = typename TileOperand<E4M3>::type;
        const unsigned char* buf = lds + at;
        const int lo = (g ^ (c & 7)) << 4, hi = ((g + 4) ^ (c & 7)) << 4;  // pieces g and g + 4
        Op w[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const unsigned char* p = buf + (w_row(i) + c) * kBlock;
            w[i] = tile_operand<E4M3>(*(const u32x4*)(p + lo), *(const u32x4*)(p + hi));
        }
        const float* wsc = (const float*)(buf + kWs);
        float ws[M];
        ws[0] = wsc[!GATED && wn * NT * 16 >= 128 ? 1 : 0] * part;
        if constexpr (GATED) ws[1] = wsc[1] * part;
        u32x4 u, v;
        float xs;
        auto fetch = [&](int t) {
            const int r = x_row(t) + c;
            const unsigned char* p = buf + kX + r * kBlock;
            u = *(const u32x4*)(p + lo);
            v = *(const u32x4*)(p + hi);
            xs = *(const float*)(buf + kXs + 4 * r);
        };
        f32x4 d[2][NT];
        float f[2][M];
        auto add = [&](int t) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[t][i][q] = __builtin_fmaf(d[t & 1][i][q], f[t & 1][GATED && i >= NT / 2 ? M - 1 : 0], acc[t][i][q]);
        };
        fetch(0);
#pragma unroll
        for (int t = 0; t < TL; ++t) {
            const Op x = tile_operand<E4M3>(u, v);
#pragma unroll
            for (int m = 0; m < M; ++m) f[t & 1][m] = xs * ws[m];
            if (t + 1 < TL) fetch(t + 1);
            tile_products(d[t & 1], w, x);
            if (E4M3) {
                add(t);
            } else {
                if (t > 0) add(t - 1);
                if (t + 1 == TL) add(t);
            }
        }
    };
    // Expert-sorted rows: tiles are seldom full, and 16 rows that are not there are left out.
    auto compute_live = [&](uint32_t at, int n, float part) {
        if (!MAPPED || x_row(MT - 1) < n) compute(Int<MT>{}, at, part);
        else if (MT > 3 && x_row(2) < n) compute(Int<(MT > 3 ? 3 : 1)>{}, at, part);
        else if (MT > 2 && x_row(1) < n) compute(Int<(MT > 2 ? 2 : 1)>{}, at, part);
        else if (MT > 1 && x_row(0) < n) compute(Int<1>{}, at, part);
    };
    // A tile's outputs (16 rows that are not there are left out, the same for the whole wave).
    auto store = [&](const RowSpan& s, int nt) {
        const int n0 = nt * kCols;
        if constexpr (!GATED) {
            const bool pairs = NT > 1 && a.out_bf16;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (x_row(t) >= s.n) break;
                const int r = x_row(t) + c;
                const size_t row = (size_t)s.row0 + r;
                if (pairs) {
                    // Two tiles of columns at once: rows of lanes trade halves, so that a lane has eight
                    // neighbours, and the four lanes of a token 64 bytes.
#pragma unroll
                    for (int i = 0; i + 1 < NT; i += 2) {
                        const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(acc[t][i][0], acc[t][i][1]),
                                                                         pack_bf16x2(acc[t][i + 1][0], acc[t][i + 1][1]), false, false);
                        const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(acc[t][i][2], acc[t][i][3]),
                                                                         pack_bf16x2(acc[t][i + 1][2], acc[t][i + 1][3]), false, false);
                        const int o = n0 + w_row(i) + 16 * (g & 1) + 8 * (g >> 1);
                        if (r < s.n) store8(a, row, o, Words<4>{{lo[0], hi[0], lo[1], hi[1]}});
                    }
                } else if (r < s.n) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) store4(a, row, n0 + w_row(i) + 4 * g, acc[t][i]);
                }
            }
        } else {
            constexpr int H = NT / 2;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (x_row(t) >= s.n) break;
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
                if (g == 0) amax[wn][x_row(t) + c] = m;
            }
            // (the next tile's first barrier lies between these reads and its writes)
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (x_row(t) >= s.n) break;
                const int r = x_row(t) + c;
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < WN; ++j) m = max(m, amax[j][r]);
                const size_t row = (size_t)s.row0 + r;
                float h[4 * H], scale;
                uint32_t codes[H];
#pragma unroll
                for (int i = 0; i < 4 * H; ++i) h[i] = acc[t][i / 4][i % 4];
                e4m3_codes<4 * H>(h, __uint_as_float(m), &scale, codes);
                if (r >= s.n) continue;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int o = n0 + w_row(i) + 4 * g;
                    if (o < N) *(uint32_t*)((uint8_t*)a.y + row * (size_t)N + o) = codes[i];
                }
                if (wn == 0 && g == 0) a.y_scale[row * (size_t)NB + nt] = scale;
            }
        }
    };

    enter(first);
#pragma unroll
    for (int j = 0; j < S - 1; ++j) load(j * kStage);
    int left = ((end - first + per_xcd - 1) / per_xcd) * KB;  // blocks still to multiply
    uint32_t here = 0;
    for (int id = first; id < end; id += per_xcd) {
        int nt;
        const RowSpan s = tile(id, &nt);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // Per block: wait for its loads (those of the next S - 2 blocks stay in flight; stores
        // that are under way only make the wait longer), start those of the block S - 1 ahead
        // into the stage that every wave has left, multiply.
        for (int b = 0; b < KB; ++b) {
            if (S > 3 && left > 2) wait_loads<(S > 3 ? 2 * kLoads : 0)>();
            else if (S > 2 && left > 1) wait_loads<(S > 2 ? kLoads : 0)>();
            else wait_loads<0>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            load(here == 0 ? (S - 1) * kStage : here - kStage);
            compute_live(here, s.n, half && b == KB - 1 ? 0.5f : 1.0f);
            here = here == (S - 1) * kStage ? 0 : here + kStage;
            --left;
        }
        store(s, nt);
    }
}

template <int BM, int BN, int WM, int WN, int S, bool E4M3, bool GATED, bool MAPPED>
void launch_tile(const ProductArgs& a, int tiles, hipStream_t s) {
    constexpr int kCols = GATED ? BN / 2 : BN;
    const long long all = (long long)tiles * ((a.N + kCols - 1) / kCols);
    constexpr int kGrid = kCus * (BN <= 64 ? 3 : S * (BM + BN) <= 600 ? 2 : 1);  // (by their LDS)
    const unsigned grid = (unsigned)(all < kGrid ? (all + 7) / 8 * 8 : kGrid);  // (some for every XCD)
    product_tile_kernel<BM, BN, WM, WN, S, E4M3, GATED, MAPPED><<<grid, WM * WN * 64, 0, s>>>(a);
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

// The largest tile that still gives every CU work: larger tiles read LDS and convert less per
// product, smaller ones fill the chip.  Measured at the borders (us):
//   experts, rows of an expert on average: gated, 2 x 512 rows, K = 2048: 32 rows 110 with tiles
//     of 32 rows and two work groups a CU, 123 with one, 131 with tiles of 128; 64 rows 157, 178
//     and 171; 128 rows 251, 292 and 232; 8 tokens (228 tiles) 25.8 and 25.1.  Not gated, tiles of
//     32 rows and of 128: 256 experts, 2048 rows, K = 512 in bf16, 24 rows 59.6 and 60.1, 32 rows
//     67.6 and 63.8, 40 rows 78 and 71, in fp32 66.8 and 64.6, 71.4 and 73.7, 87 and 76; 64 experts,
//     700 rows, K = 1088, bf16, 24 rows 14.0 and 20.2, 32 rows 22.8 and 21.7; 8 experts, 4096 x 4096,
//     24 rows 42 and 53, 32 rows 44 and 58.
//   exact products of bf16 outputs and cut ones: 64 rows, 8192 x 8192 30 and 22, 40001 x 2048 26 and
//     24; 128 rows, 4096 x 4096 16.7 and 12.7, 128256 x 4096 163 and 167; 256 rows of that 288 and
//     179; experts, 2048 rows, K = 512: 32 rows 64.8 and 58.1, 64 rows 83 and 71, 128 rows 121 and 96.
//   gated: 128 x 2 x 8192 x 2048 20 with tiles of 32 rows, 37 with 128; 512 rows 67 and 42;
//     300 x 2 x 2048 x 2048 19, 25 with 64, 36 with 128.
//   one token, 8192 x 8192: 15 in the few-token kernel, 30 in 32 x 64 tiles; 16 tokens, 16384 x
//     4096: 22 and 18.  32 tokens, 4096 x 4096: 11 and 17; 128 tokens, 2048 x 2048: 13 and 10.
//   2048 x 4096 x 4096, fp32: 79 with tiles of 128 x 128 (two work groups of four waves a CU; 88
//     with one of eight), 90 with 64 x 128; bf16: 46 (two of eight waves; one: 52, two of four:
//     50).  128 x 128 and 64 x 128: 512 rows of that, fp32 43 and 31, 1100 rows, fp32 62 and 56,
//     bf16 39 and 41.
//   The next larger of 32 x 64, 64 x 64 and 64 x 128 as soon as the smaller ones are more than the
//     CUs, fp32 / bf16: 128 x 4096 x 2048 (256 of 32 x 64) 10.3 with those and 12.0 with 64 x 64 /
//     8.2 and 9.1, 128 x 4608 x 2048 (288) 13.7 and 12.1 / 11.6 and 9.2, 128 x 5000 x 576 6.9 and
//     5.9 / 6.1 and 5.0; 64 x 16384 x 4096 (256 of 64 x 64) 21.3 with those and 25.2 with 64 x 128,
//     60 x 17000 x 4096 (266) 30.3 and 25.4, 256 x 5120 x 4096 (320) 31 and 26 / 21.4 and 18.0.
//   64 x 128, two stages and three: 512 x 4096 x 4096 in fp32 29.6 and 30.6, in bf16 24.8 and 20.5
//     (half the work between two waits).
//   Matrices that one tile of rows reads, 64 MB and more: their loads ask not to be kept (nt).  With
//     and without: gated experts, 8 tokens 23.9 and 24.7, 64 tokens 70 and 79, 512 tokens 96 and 105,
//     768 99 and 104, 1024 111 and 110; bf16, 2048 rows, K = 512, 64 tokens 37 and 43, rows of an
//     expert 8 46 and 53, 24 61 and 62, 32 69 and 65.5, and in tiles of 128 rows 40 70.6 and 72.3,
//     64 81 and 80.5, 128 106 and 95; 8 tokens, 248320 x 2048: 80 and 91.  Where tiles of rows share
//     them it costs (64 rows an expert 176 and 157), and where the last-level cache may hold them
//     from call to call (32 tokens, 2 x 8192 x 2048 gated 20 and 18).
//   8 tokens, 248320 x 2048: 91 with 32 x 256, 97 with 32 x 64; 60000 rows: 28 and 26.
hipError_t launch_product(const ProductArgs& a0, hipStream_t s) {
    ProductArgs a = a0;
    const int per = (a.rows + a.E - 1) / a.E;  // rows of an expert on average
    const bool cut = a.out_bf16 && a.rows >= 128 * a.E;  // the matrix cores' own 8-bit products
    const bool low = per <= (a.gated ? 96 : 32);  // mapped: tiles of 32 rows, else 128
    a.stream = per <= (!a.map ? 32 : low ? 24 : 64) &&
               (long long)min(a.rows, a.E) * (a.gated ? 2 : 1) * a.N * a.K >= 64ll << 20;
    auto tiles = [&](int m, int n) { return (long long)((a.rows + m - 1) / m) * ((a.N + n - 1) / n); };
    if (a.map) {
        if (low) {
            // (one tile a CU at most: all of its LDS for loads in flight)
            const bool few = (long long)min(a.rows, a.E) * ((a.N + (a.gated ? 127 : 255)) / (a.gated ? 128 : 256)) <= kCus;
            if (a.gated && few) launch_tile<32, 256, 1, 8, 4, false, true, true>(a, tiles_of<32>(a), s);
            else if (a.gated) launch_tile<32, 256, 1, 4, 2, false, true, true>(a, tiles_of<32>(a), s);
            else launch_tile<32, 256, 1, 8, 4, false, false, true>(a, tiles_of<32>(a), s);
        } else {
            if (a.gated) launch_tile<128, 256, 2, 4, 3, false, true, true>(a, tiles_of<128>(a), s);
            else if (cut) launch_tile<128, 256, 2, 4, 3, true, false, true>(a, tiles_of<128>(a), s);
            else launch_tile<128, 256, 2, 4, 3, false, false, true>(a, tiles_of<128>(a), s);
        }
    } else if (a.gated) {
        if (tiles(32, 128) <= kCus) launch_tile<32, 256, 1, 8, 4, false, true, false>(a, tiles_of<32>(a), s);
        else if (tiles(64, 128) <= kCus) launch_tile<64, 256, 1, 8, 3, false, true, false>(a, tiles_of<64>(a), s);
        else launch_tile<128, 256, 2, 4, 3, false, true, false>(a, tiles_of<128>(a), s);
    } else if (a.rows <= 16 && a.N < 16384) {
        launch_split<1>(a, s);
    } else if (tiles(32, 16) <= kCus) {
        launch_split<2>(a, s);
    } else if (a.rows > 128 && tiles(256, 256) >= kCus) {
        if (cut) launch_tile<256, 256, 2, 4, 2, true, false, false>(a, tiles_of<256>(a), s);
        else launch_tile<128, 256, 2, 4, 3, false, false, false>(a, tiles_of<128>(a), s);
    } else if (a.rows > 64 && tiles(128, 128) > kCus) {
        if (cut) launch_tile<128, 128, 2, 4, 2, true, false, false>(a, tiles_of<128>(a), s);
        else launch_tile<128, 128, 2, 2, 2, false, false, false>(a, tiles_of<128>(a), s);
    } else if (a.rows > 32 && tiles(64, 64) > kCus) {
        if (cut) launch_tile<64, 128, 2, 4, 3, true, false, false>(a, tiles_of<64>(a), s);
        else launch_tile<64, 128, 2, 4, 2, false, false, false>(a, tiles_of<64>(a), s);
    } else if (a.rows > 32 && tiles(32, 64) > kCus) {
        if (cut) launch_tile<64, 64, 2, 4, 3, true, false, false>(a, tiles_of<64>(a), s);
        else launch_tile<64, 64, 2, 4, 3, false, false, false>(a, tiles_of<64>(a), s);
    } else if (a.rows <= 32 && tiles(32, 256) >= 2 * kCus) {
        launch_tile<32, 256, 1, 8, 4, false, false, false>(a, tiles_of<32>(a), s);
    } else {
        if (cut) launch_tile<32, 64, 2, 4, 4, true, false, false>(a, tiles_of<32>(a), s);
        else launch_tile<32, 64, 2, 4, 4, false, false, false>(a, tiles_of<32>(a), s);
    }
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
