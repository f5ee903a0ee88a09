// linear.hip -- y = W x for 1 .. 64 token rows against one group-64 affine
// 4-bit matrix (moe_linear): projections and the output head of a decode step
// for several sequences or drafted tokens.
//
// Work: N K / 2 bytes of codes and N K / 16 of scales and biases, 2 T N K operations on
// the matrix cores.  With many rows (the streaming kernel) a weight is read and
// dequantised once for all T tokens (2.4 vector operations per weight), and for few
// tokens the bound is the weight stream, with the dequantisation close behind; with few
// rows (the split kernel) once for every 16 tokens.
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
//   linear_split_kernel   few rows: one or two 16-row tiles per work group, whose 16 waves
//                         share K and whose sums meet in LDS (else most CUs would idle)
//   linear_stream_kernel  many rows: every wave or pair of waves owns its tiles; x goes
//                         through LDS
// Measured (graph replays over three or four matrices in turn), for 8 / 16 / 32 / 64 tokens:
// 248320 x 2048 in 62 / 64 / 75 / 134 us (8: 4.7 TB/s), 30011 x 8192 in 39 / 44 / 52 / 69;
// 2048 x 2048 for one in 4.0, for 64 in 8.4.
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kStep = 128;  // columns per wave and step

// D of the 16x16 products: lane (c = lane & 15, g) holds token t0 + 16 n + c, rows
// row0 + 4 g .. + 3.
template <int NT>
__device__ __forceinline__ void store_tile(const LinearArgs& a, const f32x4 (&acc)[NT], int row0, int t0, int lane) {
    const int c = lane & 15, o = row0 + 4 * (lane >> 4);
    const int N = a.N;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = t0 + 16 * n + c;
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

// RT tiles of 16 rows and one of 16 tokens per work group; its 16 waves take the 128-column
// steps in turn and their sums meet in LDS in wave order.  (More tokens are more work
// groups: each dequantises its weights again, but with few rows the CUs are there, and
// what costs time is reading x, which every work group reads whole.)
constexpr int kSplitWaves = 16;

template <int RT>
__global__ __launch_bounds__(kSplitWaves * 64) void linear_split_kernel(const LinearArgs a) {
    __shared__ f32x4 red[kSplitWaves][RT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int N = a.N, K = a.K, t0 = 16 * blockIdx.y;
    const int row0 = blockIdx.x * 16 * RT;
    const int t = t0 + r < a.T ? t0 + r : a.T - 1;  // clamped, valid
    const uint16_t* xr = a.x + (size_t)t * K;
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = wave * kStep; kb < K; kb += kSplitWaves * kStep) {
        const int k0 = kb + 32 * g;
        const bool live = k0 < K;       // K is a multiple of 64: the last step may be half
        const int kk = live ? k0 : 0;   // clamped, valid
        u32x4 w[RT], x[4];
        float s9[RT], b[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int at = row0 + 16 * i + r;
            const size_t row = (size_t)(at < N ? at : N - 1);  // clamped, valid
            w[i] = *(const u32x4*)(a.w.q + row * (size_t)(K / 8) + kk / 8);
            s9[i] = live ? dq_scale(a.w.scale[row * (size_t)(K / kGroup) + kk / kGroup]) : 0.0f;
            b[i] = live ? bf16_to_f32(a.w.bias[row * (size_t)(K / kGroup) + kk / kGroup]) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = ((const u32x4*)(xr + kk))[j];
            if (!live) x[j] = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    dequant8(w[i][j], s9[i], b[i]), __builtin_bit_cast(bf16x8, x[j]), acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave >= RT) return;
    f32x4 sum[1] = {red[0][wave][lane]};
    for (int w = 1; w < kSplitWaves; ++w) sum[0] += red[w][wave][lane];
    store_tile<1>(a, sum, row0 + 16 * wave, t0, lane);
}

// Sixteen bytes at a 2-byte address (one load: the hardware takes any alignment).
struct __attribute__((packed, aligned(2))) Unaligned {
    uint32_t w[4];
};

// The 16-bit groups of v without the first n (0 <= n < 8), zeros at the end.
__device__ __forceinline__ u32x4 shift_groups(const Unaligned& v, int n) {
    uint64_t lo = v.w[0] | (uint64_t)v.w[1] << 32, hi = v.w[2] | (uint64_t)v.w[3] << 32;
    if (n & 4) {
        lo = hi;
        hi = 0;
    }
    const int s = 16 * (n & 3);
    lo = lo >> s | (hi << 1) << (63 - s);
    hi >>= s;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Many rows.  x lies in LDS as [step][16 tokens][8 columns][token] of 16 bytes: the eight
// lanes that the LDS serves at once read (r) and write (neighbouring tokens) 128
// neighbouring bytes.  NB is the number of tokens it has room for (8: lanes of tokens
// 8 .. 15 read those of 0 .. 7 again, their results are not stored).
// K goes in chunks of 512 columns, and a row's sum is two: over the first and over the
// second half of every chunk, added at the end.  The grid is one work group of 16 waves
// per CU, and the next chunk's weights, across tiles too, are loaded before the current
// chunk's products.
//   kWave     all of x (NB K 2 <= 128 KB) is staged once; after that the waves run without
//             barriers, each over its own tiles (wave w of group b: tiles w G + b, then
//             every 16 G, so that any number of tiles spreads over the CUs)
//   kPair     the same with two waves per tile, one for each half of the chunks: where
//             the tiles would leave half of the waves idle
//   kChunked  x is larger: one chunk of it at a time, double buffered, a barrier per
//             chunk; a work group's pairs of waves take eight neighbouring tiles
// Scales and biases come in blocks of 2048 columns: lane 4 i + c loads those of chunk c of
// row i (16 bytes, so 64 neighbouring bytes a row), and each product's lanes fetch theirs
// from that lane.  Loaded per chunk, 16 bytes from each of 16 rows, they cost as much time
// as the codes: the vector caches serve cache lines, not bytes (measured at N = 30011,
// K = 8192, one token: 46.5 us, and 35 without any scale loads).
// Registers: with room for 64 tokens 16 waves have too few of them in some forms.  kWave
// (K <= 1024) keeps 9 to 12 of a lane's values in scratch memory, kChunked 4 to 8 where K
// is not a multiple of 2048 (64 tokens, 40000 x 1024: 17 us; 30011 x 8128: 74 us, and
// 69 at 8192 columns).
// FULL: K is a multiple of 2048 (no branches between the loads).  VEC: of 512 (no chunk is
// cut short, a row's scales start on 16 bytes).
constexpr int kChunk = 512;
constexpr int kSteps = kChunk / kStep;
constexpr int kCus = 256;
constexpr int kThreads = 1024;
enum Mode { kWave, kPair, kChunked };

template <int NB, Mode MODE, bool FULL, bool VEC>
__global__ __launch_bounds__(kThreads) void linear_stream_kernel(const LinearArgs a) {
    constexpr int NT = (NB + 15) / 16, TB = NB < 16 ? NB : 16;
    constexpr int kStepPieces = NB * 16, kChunkPieces = NB * 64;
    constexpr int XP = MODE == kChunked ? (kChunkPieces + kThreads - 1) / kThreads : 1;  // pieces per thread
    constexpr int HS = MODE == kWave ? kSteps : kSteps / 2;  // steps of a chunk per wave
    constexpr int SUMS = MODE == kWave ? 2 : 1;
    constexpr int SLOTS = MODE == kWave ? 16 : 8;            // tiles of a work group at a time
    __shared__ u32x4 s_x[MODE == kChunked ? 2 * kChunkPieces : 8192];
    __shared__ f32x4 s_sum[MODE == kWave ? 1 : SLOTS * NT * 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int slot = wave % SLOTS, half = wave / SLOTS;
    const int r = lane & 15, g = lane >> 4;
    const int N = a.N, K = a.K, T = a.T, G = gridDim.x;
    // neighbouring units go to work groups of one XCD (group i runs on XCD i % 8), whose L2
    // joins the half lines that two tiles write
    const int b = (int)blockIdx.x, me = G % 8 == 0 ? (b & 7) * (G / 8) + (b >> 3) : b;
    // columns col .. + 7 of token t, 0 past the ends; their place in a chunk, or in x
    auto x_piece = [&](int t, int col) {
        const bool live = t < T && col < K;
        const u32x4 v = *(const u32x4*)(a.x + (live ? (size_t)t * K + col : 0));
        return live ? v : u32x4{0u, 0u, 0u, 0u};
    };
    // piece i of x or of a chunk: eight tokens, then eight neighbouring pieces of a row (128
    // bytes), then the next tokens; its place
    auto x_token = [](int i) { return (i & 7) + 8 * ((i >> 6) % (NB / 8)); };
    auto x_col = [](int i) { return ((i >> 3) & 7) + 8 * ((i >> 6) / (NB / 8)); };
    auto x_place = [&](int i) {
        const int t = x_token(i), c = x_col(i);
        return ((c >> 4) * NT + (t >> 4)) * 16 * TB + (c & 15) * TB + (t & (TB - 1));
    };
    struct Scales {
        u32x4 s, b;  // eight groups each
    };
    struct Weights {
        u32x4 q[HS];
    };
    constexpr int kUnitRows = MODE == kChunked ? 16 * SLOTS : 16;
    const int units = (N + kUnitRows - 1) / kUnitRows, stride = MODE == kChunked ? G : SLOTS * G;
    auto row_of = [&](int u) { return MODE == kChunked ? (u * SLOTS + slot) * 16 : u * 16; };
    const int st0 = half * HS;
    auto load = [&](Weights& v, int u, int kc) {
        const int row0 = row_of(u) + r;
        const size_t row = (size_t)(row0 < N ? row0 : N - 1);  // clamped, valid
        const uint32_t* qp = a.w.q + row * (size_t)(K / 8);
#pragma unroll
        for (int st = 0; st < HS; ++st) {
            const int k0 = kc + (st0 + st) * kStep + 32 * g, kk = VEC && FULL || k0 < K ? k0 : 0;  // clamped, valid
            v.q[st] = *(const u32x4*)(qp + kk / 8);
        }
    };
    // the scales of the 2048 columns from kb on (groups past the row's end: its last)
    auto load_scales = [&](Scales& v, int u, int kb) {
        const int row0 = row_of(u) + (lane >> 2);
        const int groups = K / kGroup, g0 = kb / kGroup + 8 * (lane & 3);
        const size_t so = (size_t)(row0 < N ? row0 : N - 1) * (size_t)groups;  // clamped, valid
        if constexpr (VEC) {
            const size_t o = so + (FULL || g0 < groups ? g0 : 0);
            v.s = *(const u32x4*)(a.w.scale + o);
            v.b = *(const u32x4*)(a.w.bias + o);
        } else {
            // eight groups from any 2-byte address, inside the array (it has eight at least);
            // where that starts before g0, the first ones are shifted out
            const size_t o = so + min(g0, groups - 1), end = (size_t)N * groups - 8, at = o < end ? o : end;
            v.s = shift_groups(*(const Unaligned*)(a.w.scale + at), (int)(o - at));
            v.b = shift_groups(*(const Unaligned*)(a.w.bias + at), (int)(o - at));
        }
    };
    f32x4 acc[SUMS][NT];
    auto clear = [&] {
#pragma unroll
        for (int h = 0; h < SUMS; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[h][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    // One chunk.  The operands of x for product q + 1 are read before the weights of
    // product q are dequantised, so that their latency runs under that.
    auto products = [&](const Weights& v, const Scales& sc, int c, const u32x4* x, int kc) {
        const u32x4* xl = x + st0 * kStepPieces + 4 * g * TB + (r & (TB - 1));
        const int steps = VEC ? HS : max(0, min(HS, (K - kc + kStep - 1) / kStep - st0));
        // word st0 + st of the chunk's scales holds the step's two groups
        uint32_t sw[HS], bw[HS];
#pragma unroll
        for (int st = 0; st < HS; ++st) {
            const uint32_t s = HS == 4 ? sc.s[st] : half ? sc.s[2 + st] : sc.s[st];
            const uint32_t b = HS == 4 ? sc.b[st] : half ? sc.b[2 + st] : sc.b[st];
            sw[st] = (uint32_t)__builtin_amdgcn_ds_bpermute(16 * r + 4 * c, (int)s);
            bw[st] = (uint32_t)__builtin_amdgcn_ds_bpermute(16 * r + 4 * c, (int)b);
        }
        // (four operands of two products do not fit the registers of 16 waves: read for the
        // same product then, ahead of its dequantisation)
        constexpr int AHEAD = NT == 4 ? 0 : 1;
        u32x4 xo[1 + AHEAD][NT];
        if (AHEAD && (VEC || steps > 0)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) xo[0][n] = xl[n * 16 * TB];
        }
        float s9 = 0.0f, bi = 0.0f;
#pragma unroll
        for (int q = 0; q < 4 * HS; ++q) {
            const int st = q >> 2, j = q & 3, h = SUMS == 2 ? st >> 1 : 0;
            if (!VEC && st >= steps) break;  // uniform
            if (q + AHEAD < 4 * HS && (!AHEAD || VEC || j < 3 || st + 1 < steps)) {
                const int qa = q + AHEAD;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    xo[qa & AHEAD][n] = xl[(qa >> 2) * kStepPieces + n * 16 * TB + (qa & 3) * TB];
            }
            __builtin_amdgcn_sched_barrier(0);
            if (j == 0) {  // group 2 st + (g >> 1): one half of the word
                const int up = g & 2 ? 0 : 16;
                s9 = __uint_as_float((sw[st] << up) & 0xFFFF0000u) * 512.0f;
                bi = __uint_as_float((bw[st] << up) & 0xFFFF0000u);
                if (!VEC && kc + (st0 + st) * kStep + 32 * g >= K) s9 = bi = 0.0f;  // half a step
            }
            const bf16x8 wv = dequant8(v.q[st][j], s9, bi);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[h][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    wv, __builtin_bit_cast(bf16x8, xo[q & AHEAD][n]), acc[h][n], 0, 0, 0);
        }
    };
    int u = MODE == kChunked ? me : slot * G + me, buf = 0;
    const int u_first = u;
    Weights w0, w1;
    Scales sc, sc_next;
    load_scales(sc, u, 0);
    load(w0, u, 0);
    clear();
    if constexpr (MODE == kChunked) {
#pragma unroll
        for (int p = 0; p < XP; ++p) {
            const int i = tid + p * kThreads;
            if (i < kChunkPieces) s_x[x_place(i)] = x_piece(x_token(i), 8 * x_col(i));
        }
    } else {
        const int pieces = (K + kStep - 1) / kStep * kStepPieces;
        for (int i = tid; i < pieces; i += kThreads) s_x[x_place(i)] = x_piece(x_token(i), 8 * x_col(i));
    }
    __syncthreads();
    // Chunk c of the block at kb with `cur`, while the next chunk is loaded to `nxt`.  (Loads
    // are made whether they will be used or not, from a valid place: with the loads in a
    // branch the compiler cannot count those in flight and waits for all of them.)
    auto chunk = [&](int c, int kb, int u2, const Weights& cur, Weights& nxt) {
        const int kc = kb + c * kChunk;
        const bool last = kc + kChunk >= K;
        const bool dummy = !FULL && kc >= K;  // uniform; evens the number of chunks
        const bool block_end = c == 3 || (!FULL && c == 1 && kc + kChunk >= K);
        const int un = block_end ? u2 : u, kn = block_end ? (kb + 2048 < K ? kb + 2048 : 0) : kc + kChunk;
        load(nxt, un, kn);
        u32x4 xn[XP];
        if constexpr (MODE == kChunked) {
#pragma unroll
            for (int p = 0; p < XP; ++p) {
                const int i = tid + p * kThreads;
                xn[p] = x_piece(x_token(i), kn + 8 * x_col(i));
            }
        }
        if (!dummy)
            products(cur, sc, c, MODE == kChunked ? s_x + buf * kChunkPieces : s_x + kc / kStep * kStepPieces,
                     kc);
        if (MODE == kWave && last && !dummy) {
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[0][n] += acc[SUMS - 1][n];
            store_tile<NT>(a, acc[0], row_of(u), 0, lane);
            clear();
        }
        if constexpr (MODE == kChunked) {
            if (last && !dummy && half == 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s_sum[(slot * NT + n) * 64 + lane] = acc[0][n];
            }
            buf ^= 1;  // (read last before the previous barrier)
#pragma unroll
            for (int p = 0; p < XP; ++p) {
                const int i = tid + p * kThreads;
                if (i < kChunkPieces) s_x[buf * kChunkPieces + x_place(i)] = xn[p];
            }
            __syncthreads();
            if (last && !dummy) {
                if (half == 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[0][n] += s_sum[(slot * NT + n) * 64 + lane];
                    store_tile<NT>(a, acc[0], row_of(u), 0, lane);
                }
                clear();
                // (s_sum is written again after another barrier at least: a tile has an even
                // number of chunks, dummies included)
            }
        }
    };
    int kb = 0;
    while (u < units) {  // (by wave; kChunked: by work group)
        const bool row_end = kb + 2048 >= K;
        const int u2 = row_end ? u + stride : u, kb2 = row_end ? 0 : kb + 2048;
        load_scales(sc_next, u2, kb2);
        chunk(0, kb, u2, w0, w1);
        chunk(1, kb, u2, w1, w0);
        if (FULL || kb + 2 * kChunk < K) {
            chunk(2, kb, u2, w0, w1);
            chunk(3, kb, u2, w1, w0);
        }
        sc = sc_next;
        u = u2;
        kb = kb2;
    }
    if constexpr (MODE == kPair) {  // (one tile per pair)
        if (u_first < units && half == 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n) s_sum[(slot * NT + n) * 64 + lane] = acc[0][n];
        }
        __syncthreads();
        if (u_first < units && half == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[0][n] += s_sum[(slot * NT + n) * 64 + lane];
            store_tile<NT>(a, acc[0], row_of(u_first), 0, lane);
        }
    }
}

template <int NB, Mode MODE>
void launch_stream(const LinearArgs& a, hipStream_t s) {
    const int tiles = (a.N + 15) / 16, units = MODE == kChunked ? (tiles + 7) / 8 : tiles;
    const int grid = units < kCus ? units : kCus;
    if constexpr (MODE == kChunked || NB <= 32) {  // (64 tokens of 2048 columns do not fit the LDS)
        if (a.K % 2048 == 0) {
            linear_stream_kernel<NB, MODE, true, true><<<grid, kThreads, 0, s>>>(a);
            return;
        }
    }
    if (a.K % kChunk == 0) linear_stream_kernel<NB, MODE, false, true><<<grid, kThreads, 0, s>>>(a);
    else linear_stream_kernel<NB, MODE, false, false><<<grid, kThreads, 0, s>>>(a);
}

// By rows, from both sides' times (us; the choice has to go by N and K alone, so that T
// tokens give the bits of T single ones).  At 4096 rows, one token / 64 tokens, split with
// one tile and streamed: K = 512 2.9 / 5.9 and 3.6 / 6.2, 2048 4.2 / 14.7 and 5.9 / 17.2,
// 8192 9.6 / 51 and 15.8 / 56.  At 6000, split with two tiles and streamed: 3.3 / 6.4 and
// 3.6 / 6.3, 6.2 / 16.4 and 6.2 / 17.9, 15.7 / 55 and 16.9 / 56.  At 8192: 3.4 / 7.2 and
// 3.7 / 6.5, 6.6 / 20.8 and 6.3 / 18.3, 15.9 / 72 and 17.1 / 57.  Pairs of waves against one
// wave a tile, 16384 rows, one token: 4.0 and 4.3, 7.0 and 7.9, 20.6 and 22.2.
template <int NB>
void launch(const LinearArgs& a, hipStream_t s) {
    const bool fits = NB * ((a.K + kStep - 1) / kStep) <= 512;  // x in 128 KB
    const int groups = (a.T + 15) / 16, tiles = (a.N + 15) / 16;
    if (a.N <= 4096) linear_split_kernel<1><<<dim3(tiles, groups), kSplitWaves * 64, 0, s>>>(a);
    else if (a.N < 8192) linear_split_kernel<2><<<dim3((tiles + 1) / 2, groups), kSplitWaves * 64, 0, s>>>(a);
    else if (fits && a.N <= 16 * 8 * kCus) launch_stream<NB, kPair>(a, s);
    else if (fits) launch_stream<NB, kWave>(a, s);
    else if constexpr (NB > 8) launch_stream<NB, kChunked>(a, s);
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
