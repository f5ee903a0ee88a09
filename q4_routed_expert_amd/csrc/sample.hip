// sample.hip -- one token per row of logits: temperature, top-k, top-p, min-p and
// a draw from a given uniform number (moe_sample).
//
// Order of a row's tokens: larger logit first, equal logits by the lower index; all
// three filters keep a prefix of that order.  Weights are
//   w_i = round(2^43 exp(-x_i)),  x_i = (l_max - l_i) / temperature < 30.4
// (0 beyond, where the rounding gives at most 1) as 64-bit integers, so every sum is
// exact (V <= 2^20 weights of at most 2^43) and the same in any order: atomics and
// split sums give the same token every time, and a weight's rounding, 2^-44 of the
// largest, is far below the step of a 24-bit uniform number.  Only the drawn token's
// probability takes its weight unrounded: a rounding of 2^-44 is 2^-19 of a weight at
// depth 17, more than fp32 keeps.
//
// The draw runs over the kept tokens in index order, so nothing is ever sorted: all
// that is needed of the order is its cut, the last kept token.  It is the first at
// which a running quantity reaches a target: the count reaches top_k, or the mass
// reaches top_p of the sum.  A histogram of that quantity over 2048 bins of x gives
// the bin it falls into, and the few tokens of that bin are ranked among each other.
//
// Long rows (four kernels, the first three over B x C chunks of the logits):
//   1. sample_max_kernel     largest logit of every chunk; clears the row's histogram
//   2. sample_hist_kernel    the histogram (counts with top-k: no exponentials at all)
//   3. sample_gather_kernel  the cut's bin; its tokens into the row's list (with top-k:
//                            all tokens down to that bin), each chunk's mass before it
//   4. sample_pick_kernel    one work group per row: the exact cut, the chunk that holds
//                            the drawn mass, the token in it, its embedding row
// A row without top-k and top-p needs no cut: kernel 2 writes the chunks' masses
// itself.  If the list overflows (more than 4096 tokens, or 2048 of one chunk), kernel 4
// narrows over the whole row instead, some 70 us a pass at V = 248320.  That takes
// thousands of equal logits at the cut, a top-k in the thousands, or a flat row under
// top-p: a bin is 0.0148 wide, and 248320 normal logits of spread / temperature 0.36 put
// 4096 into the one at their middle (one row and 64 rows of 248320: 0.13 and 0.35 ms at
// 0.2 with top-p 0.9, 0.38 and 0.36 with top-k 20000; all logits equal, one row: 0.58).
// Short rows (sample_row_kernel): one work group does all of it with the row in its
// registers.
#include <float.h>

#include "ops.h"

namespace q4moe {
namespace {

constexpr int kThreads = 512;       // of kernels 1 to 3
constexpr int kRowThreads = 1024;   // of kernel 4 and of the short rows' kernel, at most
constexpr int kBins = kSampleBins;
constexpr int kList = kSampleList;
constexpr int kRank = 256;          // tokens ranked against each other at once
constexpr int kMaxChunks = kSampleMaxChunks;
constexpr int kIdxBits = 20;        // MOE_MAX_VOCAB = 2^20
constexpr double kOne = 8796093022208.0;  // 2^43: the weight of the largest logit
constexpr double kRange = 30.4;           // beyond this depth a weight is 0

// One row's parameters from the caller's arrays.
__device__ __forceinline__ SampleRow row_params(const SampleArgs& a, int b) {
    float t = a.temperature_all, p = a.top_p_all, mp = a.min_p_all;
    int k = a.top_k_all;
    if (a.temperature) t = a.temperature[b];  // all the loads before any use
    if (a.top_k) k = a.top_k[b];
    if (a.top_p) p = a.top_p[b];
    if (a.min_p) mp = a.min_p[b];
    SampleRow r;
    r.u = a.u[b];
    const bool greedy = !(t > 0.0f);
    r.inv_t = greedy ? 1.0 : 1.0 / (double)t;
    r.k = greedy ? 1u : (k <= 0 || k > a.V) ? (uint32_t)a.V : (uint32_t)k;
    r.cut_k = r.k < (uint32_t)a.V;
    r.cut_p = p < 1.0f && !greedy;
    r.p = p > 0.0f ? (double)p : 0.0;
    mp = mp > 0.0f ? fminf(mp, 1.0f) : 0.0f;  // (NaN: off)
    const double m = ceil((double)mp * kOne);
    r.w_min = m < 1.0 ? 1ull : (uint64_t)m;
    return r;
}

// Mass that top-p has to reach: at least 1, so that the first token is kept.
__device__ __forceinline__ uint64_t p_target(double p, uint64_t total) {
    const double t = ceil(p * (double)total);
    return t < 1.0 ? 1ull : (uint64_t)t;
}

// Depth x of a logit below the row's largest: 0 .. infinity, or NaN for a NaN logit (and
// for 0 * infinity, which a masked logit gives at the temperature infinity).  Infinite
// logits count as the largest finite value; m is finite.
__device__ __forceinline__ double depth(float l, double m, double inv_t) {
    return (m - (double)(l > FLT_MAX ? FLT_MAX : l)) * inv_t;
}

// Adding 1.5 * 2^52 to a double of moderate size leaves the nearest integer in the low
// bits of the sum: no conversion instruction.
constexpr double kMagic = 6755399441055744.0;
__device__ __forceinline__ int magic_int(double v) { return (int)(uint32_t)(uint64_t)__double_as_longlong(v); }

// Bin of a depth below kRange; deeper logits have higher bins (the nearest integer, so
// bin 0 is half as wide as the others).  Depths start at 0; the unsigned minimum keeps
// the index inside the histogram also where the logits change under the call, so that
// the maximum that was read is not theirs.
__device__ __forceinline__ int bin_of(double x) {
    return (int)min((uint32_t)kBins - 1, (uint32_t)magic_int(__builtin_fma(x, kBins / kRange, kMagic)));
}

// 2^43 exp(-x) for 0 <= x < kRange.  x = n ln 2 - r with |r| <= ln 2 / 2; exp(r) =
// 1 + r g(r), g the polynomial of degree 8 through (exp(r) - 1) / r at the nine Chebyshev
// nodes of the interval (relative error below 2^-44 = half a unit of the largest
// weight); 2^(43 - n) by the exponent field.  Only full-rate 64-bit arithmetic.
__device__ __forceinline__ double exp_in(double x) {
    const double t = fma_const(x, 1.4426950408889634, kMagic);
    const double n = t - kMagic;
    const double r = __builtin_fma(n, 0.69314718055994529, -x);
    double e = 2.7625104765945114e-06;
    e = fma_const(e, r, 2.487616679288376e-05);
    e = fma_const(e, r, 0.00019841208751916224);
    e = fma_const(e, r, 0.0013888821672636716);
    e = fma_const(e, r, 0.008333333353719753);
    e = fma_const(e, r, 0.04166666689098201);
    e = fma_const(e, r, 0.166666666666483);
    e = fma_const(e, r, 0.49999999999797906);
    e = __builtin_fma(e, r, 1.0);
    e = __builtin_fma(e, r, 1.0);
    return __longlong_as_double((long long)((uint64_t)__double_as_longlong(e) +
                                            ((uint64_t)(uint32_t)(43 - magic_int(t)) << 52)));
}

// Its rounding: adding 2^52 leaves the integer in the low bits of the sum.
__device__ __forceinline__ uint64_t weight_in(double x) {
    return (uint64_t)__double_as_longlong(exp_in(x) + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;
}

// The weight at any depth: 0 beyond the range and for NaN.
__device__ __forceinline__ uint64_t weight_at(double x) { return x < kRange ? weight_in(x) : 0; }

__device__ __forceinline__ uint64_t weight(float l, double m, double inv_t) {
    return weight_at(depth(l, m, inv_t));
}

// A token's place in the row's order as one number: larger is earlier.
__device__ __forceinline__ uint64_t place(float l, int i) {
    return ((uint64_t)logit_key(l) << kIdxBits) | (uint32_t)((1 << kIdxBits) - 1 - i);
}
__device__ __forceinline__ int place_index(uint64_t p) {
    return (1 << kIdxBits) - 1 - (int)(p & ((1 << kIdxBits) - 1));
}
__device__ __forceinline__ float place_logit(uint64_t p) { return key_logit((uint32_t)(p >> kIdxBits)); }

// Wave-wide operations on the vector ALUs (DPP), without the LDS round trips of
// shuffles.
__device__ __forceinline__ float wave_max_f(float v) {  // (NaN is passed over)
    v = fmaxf(v, dpp_f32<0xB1>(v));   // quad_perm 1,0,3,2
    v = fmaxf(v, dpp_f32<0x4E>(v));   // quad_perm 2,3,0,1
    v = fmaxf(v, dpp_f32<0x141>(v));  // row_half_mirror
    v = fmaxf(v, dpp_f32<0x140>(v));  // row_mirror
    auto lane = [&](int i) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i)); };
    return fmaxf(fmaxf(lane(0), lane(16)), fmaxf(lane(32), lane(48)));
}

// The value kCtrl moves to this lane, 0 where it moves none (rows not in kRows).
template <int kCtrl, int kRows>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, kCtrl, kRows, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), kCtrl, kRows, 0xF, true);
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ uint64_t readlane_u64(uint64_t v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return ((uint64_t)hi << 32) | lo;
}

// Inclusive running sum over the wave's lanes: within rows of 16, then each row's total
// to the next one (rows 1 and 3), then row 1's total to rows 2 and 3.
__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t v) {
    v += dpp_u64<0x111, 0xF>(v);  // row_shr 1
    v += dpp_u64<0x112, 0xF>(v);
    v += dpp_u64<0x114, 0xF>(v);
    v += dpp_u64<0x118, 0xF>(v);
    v += dpp_u64<0x142, 0xA>(v);  // row_bcast 15
    v += dpp_u64<0x143, 0xC>(v);  // row_bcast 31
    return v;
}

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) { return readlane_u64(wave_scan_u64(v), 63); }

// Largest of the wave (0 is the smallest value), returned to every lane.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    auto step = [&](uint64_t o) { v = o > v ? o : v; };
    step(dpp_u64<0x111, 0xF>(v));
    step(dpp_u64<0x112, 0xF>(v));
    step(dpp_u64<0x114, 0xF>(v));
    step(dpp_u64<0x118, 0xF>(v));
    step(dpp_u64<0x142, 0xA>(v));
    step(dpp_u64<0x143, 0xC>(v));
    return readlane_u64(v, 63);
}

// Sum over the work group, returned to every thread.  s holds one entry per wave.
template <int NT>
__device__ __forceinline__ uint64_t group_sum_u64(uint64_t v, uint64_t* s) {
    v = wave_sum_u64(v);
    __syncthreads();  // s may still be read from the previous use
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) t += s[w];
    return t;
}

template <int NT>
__device__ __forceinline__ float group_max_f(float m, float* s) {
    m = wave_max_f(m);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
    __syncthreads();
    m = s[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, s[w]);
    return m;
}

// The row's largest logit from the chunks', by every wave for itself; infinity as the
// largest finite value.  -infinity: no live logit (then every depth is NaN or infinite).
__device__ __forceinline__ double row_max(const SampleArgs& a, int b) {
    const float* part = a.part_max + (size_t)b * a.n_chunks;
    float m = -INFINITY;
    for (int c = threadIdx.x & 63; c < a.n_chunks; c += 64) m = fmaxf(m, part[c]);
    return (double)fminf(wave_max_f(m), FLT_MAX);
}

// This thread's logits of the range [i0, i1) of row b, kPieces aligned 16-byte pieces at
// a time (aligned whatever V is: a piece at an end of the range may hold elements outside
// it, which read as minus infinity, and the piece that would cross the end of the whole
// array is read element by element).
constexpr int kPieces = 4;
__device__ __forceinline__ f32x4 load_piece(const float* p, int64_t g, int64_t n) {
    if (4 * g + 4 <= n) return *(const f32x4*)(p + 4 * g);
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 4 * g + j < n ? p[4 * g + j] : 0.0f;
    return v;
}
// Elements base .. base + 3 of which those outside [i0, i1) become minus infinity.
__device__ __forceinline__ void mask_piece(f32x4& v, int base, int i0, int i1) {
    if (base >= i0 && base + 4 <= i1) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (base + j < i0 || base + j >= i1) v[j] = -INFINITY;
}
struct Logits {
    const float* p;     // the array
    int64_t o, g1, n;   // the row's first element, the range's last piece + 1, the array's size
    int i0, i1;
    int64_t g;          // this thread's next piece
    f32x4 v[kPieces];

    __device__ __forceinline__ Logits(const SampleArgs& a, int b, int from, int to)
        : p(a.logits), o((int64_t)b * a.V), n((int64_t)a.B * a.V), i0(from), i1(to) {
        g = ((o + i0) >> 2) + threadIdx.x;
        g1 = (o + i1 + 3) >> 2;
        load();
    }
    __device__ __forceinline__ void load() {
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int64_t at = g + u * kThreads;
            if (at < g1) v[u] = load_piece(p, at, n);
        }
    }
    // f(logit, index) for all of them; the first pieces were loaded by the constructor
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        while (g < g1) {
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                const int64_t at = g + u * kThreads;
                if (at >= g1) break;
                const int base = (int)(4 * at - o);
                mask_piece(v[u], base, i0, i1);
#pragma unroll
                for (int j = 0; j < 4; ++j) f(v[u][j], base + j);
            }
            g += kPieces * kThreads;
            load();
        }
    }
};

__global__ __launch_bounds__(kThreads) void sample_max_kernel(const SampleArgs a) {
    __shared__ float s[kThreads / 64];
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    // the row's histogram and counter, shared out over its chunks
    for (int i = c * kThreads + tid; i < kBins; i += a.n_chunks * kThreads) a.hist[(size_t)b * kBins + i] = 0;
    if (c == 0 && tid == 0) {
        a.list_n[b] = 0;
        a.row[b] = row_params(a, b);
    }
    const int i0 = c << a.chunk_sh;
    Logits in(a, b, i0, min(a.V, i0 + (1 << a.chunk_sh)));
    float m = -INFINITY;
    in.each([&](float l, int) { m = fmaxf(m, l); });  // (NaN is passed over)
    m = group_max_f<kThreads>(m, s);
    if (tid == 0) a.part_max[(size_t)b * a.n_chunks + c] = m;
}

__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const SampleArgs a) {
    __shared__ unsigned long long s_h[kBins];
    __shared__ uint64_t s_sum[kThreads / 64];
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const int i0 = c << a.chunk_sh;
    Logits in(a, b, i0, min(a.V, i0 + (1 << a.chunk_sh)));  // its first loads go ahead of all else
    const SampleRow p = a.row[b];
    const double m = row_max(a, b);
    if (!p.cut_k && !p.cut_p) {  // uniform over the work group
        uint64_t sum = 0;
        in.each([&](float l, int) {
            const uint64_t w = weight(l, m, p.inv_t);
            sum += w >= p.w_min ? w : 0;
        });
        sum = group_sum_u64<kThreads>(sum, s_sum);
        if (tid == 0) a.chunk_w[(size_t)b * a.n_chunks + c] = sum;
        return;
    }
    for (int i = tid; i < kBins; i += kThreads) s_h[i] = 0;
    __syncthreads();
    if (p.cut_k) {  // (two loops: the choice stays out of them)
        in.each([&](float l, int) {
            const double x = depth(l, m, p.inv_t);
            if (x < kRange) atomicAdd(&s_h[bin_of(x)], 1ull);
        });
    } else {
        in.each([&](float l, int) {
            const double x = depth(l, m, p.inv_t);
            if (x < kRange) atomicAdd(&s_h[bin_of(x)], (unsigned long long)weight_in(x));
        });
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads)
        if (s_h[i]) atomicAdd((unsigned long long*)&a.hist[(size_t)b * kBins + i], s_h[i]);
}

// First of the kBins bins at which the running sum reaches the target (of(total) gives
// it); bin = kBins if none does.  Called by all NT threads.
struct Cut {
    int bin;
    uint64_t before;  // the sum before the bin
    uint64_t here;    // the bin's value
    uint64_t total;
};
struct CutScratch {
    uint64_t wave[kRowThreads / 64];
    Cut cut;
};

template <int NT, typename Of>
__device__ __forceinline__ Cut find_cut(const uint64_t* h, CutScratch& s, Of of) {
    constexpr int PER = kBins / NT;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t v[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        v[j] = h[tid * PER + j];
        sum += v[j];
    }
    const uint64_t inc = wave_scan_u64(sum);
    __syncthreads();  // the scratch may still be read from the previous use
    if (lane == 63) s.wave[wave] = inc;
    if (tid == 0) s.cut.bin = kBins;
    __syncthreads();
    uint64_t run = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        run += w < wave ? s.wave[w] : 0;
        total += s.wave[w];
    }
    const uint64_t target = of(total);
#pragma unroll
    for (int j = 0; j < PER; ++j) {  // exactly one thread sees the first crossing, if any
        if (run < target && run + v[j] >= target) s.cut = Cut{tid * PER + j, run, v[j], total};
        run += v[j];
    }
    __syncthreads();
    Cut c = s.cut;
    c.total = total;
    return c;
}

__global__ __launch_bounds__(kThreads) void sample_gather_kernel(const SampleArgs a) {
    constexpr uint32_t kLocal = 2048;  // entries of the list that one chunk may give
    __shared__ unsigned long long s_list[kLocal];
    __shared__ uint32_t s_n, s_base;
    __shared__ uint64_t s_sum[kThreads / 64];
    __shared__ CutScratch s_cut;
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const SampleRow p = a.row[b];
    if (!p.cut_k && !p.cut_p) return;  // uniform
    const int i0 = c << a.chunk_sh;
    Logits in(a, b, i0, min(a.V, i0 + (1 << a.chunk_sh)));
    const double m = row_max(a, b);
    // with top-k the list takes every token down to the bin of the last one it keeps
    // (top-p's mass is a share of what top-k keeps, so both cuts lie in there); if top-k
    // keeps every token with a weight, that is all of them.  top-p alone: only the bin
    // in which the mass is reached.
    const Cut cut = find_cut<kThreads>(a.hist + (size_t)b * kBins, s_cut, [&](uint64_t total) {
        return p.cut_k ? (uint64_t)p.k : p_target(p.p, total);
    });
    const int hi = min(cut.bin, kBins - 1), lo = p.cut_k ? 0 : hi;
    if (c == 0 && tid == 0)
        a.state[b] = SampleState{cut.total, p.cut_k ? 0 : cut.before, lo, hi, cut.bin < kBins, 0};
    if (tid == 0) s_n = 0;
    __syncthreads();
    uint64_t sum = 0;
    in.each([&](float l, int i) {
        const double x = depth(l, m, p.inv_t);
        if (!(x < kRange)) return;
        const int bin = bin_of(x);
        if (bin < lo) {
            const uint64_t w = weight_in(x);
            sum += w >= p.w_min ? w : 0;
        } else if (bin <= hi) {
            const uint32_t at = atomicAdd(&s_n, 1u);
            if (at < kLocal) s_list[at] = place(l, i);
        }
    });
    sum = group_sum_u64<kThreads>(sum, s_sum);  // (its barriers also complete the list)
    // a list that overflows, in a chunk or in all, is not used: list_n says so
    const uint32_t n = s_n <= kLocal ? s_n : (uint32_t)kList + 1;
    if (tid == 0) {
        a.chunk_w[(size_t)b * a.n_chunks + c] = sum;
        s_base = n ? atomicAdd(&a.list_n[b], n) : 0;
    }
    __syncthreads();
    if (n > kLocal) return;
    for (uint32_t i = tid; i < n; i += kThreads)
        if (s_base + i < (uint32_t)kList) a.list[(size_t)b * kList + s_base + i] = s_list[i];
}

// Shared memory of the work group that makes a row's cut and draw.
struct Draw {
    uint64_t hist[kBins];
    ulonglong2 rank[kRank];  // (place, weight) of the tokens that are ranked
    unsigned long long lo, hi, cut, cut_k, mass;
    uint32_t n;
    CutScratch cs;
    uint64_t sum[kRowThreads / 64];
    float m[kRowThreads / 64];
    int token;
    float logit;  // the token's
};

// Collects the region's tokens with lo <= place <= hi for ranking; false if there are
// more than kRank.  s.n has to be 0 before; a barrier completes it here.
template <typename Each>
__device__ __forceinline__ bool collect(Draw& s, uint64_t lo, uint64_t hi, Each each) {
    each([&](uint64_t p, auto q) {
        if (p >= lo && p <= hi && s.n <= (uint32_t)kRank) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < (uint32_t)kRank) s.rank[at] = ulonglong2{p, q()};
        }
    });
    __syncthreads();
    return s.n <= (uint32_t)kRank;
}

// Ranks the n collected tokens by comparing each with each: 2^sh threads a token, as many
// as the work group has.  leader: this thread holds the result for token *me, of which
// *count tokens with the mass *mass lie before.
template <int NT>
__device__ __forceinline__ bool rank_tokens(const Draw& s, int n, ulonglong2* me, uint32_t* count,
                                            uint64_t* mass) {
    const int tid = threadIdx.x;
    int sh = 0;
    while (sh < 5 && (n << (sh + 1)) <= NT) ++sh;
    const int i = tid >> sh, q = 1 << sh, part = tid & (q - 1);
    const ulonglong2 mine = s.rank[i < n ? i : 0];
    uint32_t c = 0;
    uint64_t w = 0;
    if (i < n) {
#pragma unroll 4
        for (int j = part; j < n; j += q) {
            const ulonglong2 o = s.rank[j];
            const bool before = o.x > mine.x;
            c += before;
            w += before ? o.y : 0;
        }
    }
    for (int o = 1; o < q; o <<= 1) {
        c += __shfl_xor(c, o, kWave);
        w += __shfl_xor(w, o, kWave);
    }
    *me = mine;
    *count = c;
    *mass = w;
    return i < n && part == 0;
}

// The last kept token of a region: the first, in the row's order, at which the running
// sum of a quantity reaches the target (some token does).  each(f) calls f(place, q) for
// this thread's tokens of the region; q() is the quantity, computed only where it is
// asked for.  Tokens are narrowed down by their
// place, a factor of 2048 a time, until kRank of them are left, which are ranked.
// Returns the token's place.
template <int NT, typename Each>
__device__ __forceinline__ uint64_t narrow_cut(Draw& s, uint64_t target, Each each) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) {
        s.cut = 0;  // (not reached: everything is kept)
        s.lo = ~0ull;
        s.hi = 0;
    }
    __syncthreads();
    uint64_t l = 0, h = 0;  // ~smallest and largest place (0: no token)
    each([&](uint64_t p, auto) {
        l = ~p > l ? ~p : l;
        h = p > h ? p : h;
    });
    l = ~wave_max_u64(l);
    h = wave_max_u64(h);
    if ((tid & 63) == 0 && h >= l) {
        atomicMin(&s.lo, l);
        atomicMax(&s.hi, h);
    }
    __syncthreads();
    uint64_t lo = s.lo, hi = s.hi;
    if (hi < lo) return 0;  // (uniform; no tokens at all)
    for (;;) {
        const int bits = hi > lo ? 64 - __builtin_clzll(hi - lo) : 0;
        const int shift = bits > 11 ? bits - 11 : 0;
        for (int i = tid; i < kBins; i += NT) s.hist[i] = 0;
        if (tid == 0) s.n = 0;
        __syncthreads();
        each([&](uint64_t p, auto q) {
            if (p >= lo && p <= hi)
                atomicAdd((unsigned long long*)&s.hist[(int)((hi - p) >> shift)], (unsigned long long)q());
        });
        __syncthreads();
        const Cut c = find_cut<NT>(s.hist, s.cs, [&](uint64_t) { return target; });
        if (c.bin >= kBins) return 0;
        target -= c.before;
        hi -= (uint64_t)c.bin << shift;
        if (shift == 0) return hi;
        const uint64_t bottom = hi - ((1ull << shift) - 1);
        lo = bottom > lo ? bottom : lo;
        if (collect(s, lo, hi, each)) {
            ulonglong2 me;
            uint32_t count;
            uint64_t run;
            if (rank_tokens<NT>(s, (int)s.n, &me, &count, &run) && run < target && run + me.y >= target)
                s.cut = me.x;
            __syncthreads();
            return s.cut;
        }
        __syncthreads();  // s.n is read above and cleared in the next round
    }
}

// The cut of a row whose region's tokens each(f) visits as f(place, weight()): top-k (if
// its target lies in the region), then top-p.  base: mass before the region, total: the
// mass top-p refers to without top-k.  few: the region may hold kRank tokens or fewer.
template <int NT, typename Each>
__device__ __forceinline__ uint64_t row_cut(Draw& s, const SampleRow& p, bool k_reached, uint64_t base,
                                            uint64_t total, bool few, Each each) {
    const int tid = threadIdx.x;
    if (few) {
        if (tid == 0) {
            s.n = 0;
            s.cut = s.cut_k = 0;
            s.mass = 0;
        }
        __syncthreads();
        if (collect(s, 0, ~0ull, each)) {  // one ranking serves both cuts
            const int n = (int)s.n;
            ulonglong2 me;
            uint32_t count;
            uint64_t run;
            const bool leader = rank_tokens<NT>(s, n, &me, &count, &run);
            if (p.cut_k) {
                // the last token that top-k keeps and the mass up to it
                if (leader && count + 1 == min(p.k, (uint32_t)n)) {
                    s.cut_k = k_reached ? me.x : 0;
                    s.mass = run + me.y;
                }
                __syncthreads();
                if (!p.cut_p) return s.cut_k;
                total = s.mass;
                base = 0;
            }
            const uint64_t target = p_target(p.p, total) - base;
            if (leader && run < target && run + me.y >= target) s.cut = me.x;
            __syncthreads();
            return p.cut_k && s.cut_k > s.cut ? s.cut_k : s.cut;
        }
    }
    uint64_t last = 0;
    if (p.cut_k) {
        if (k_reached)
            last = narrow_cut<NT>(s, p.k, [&](auto f) { each([&](uint64_t pl, auto) { f(pl, [] { return 1ull; }); }); });
        if (!p.cut_p) return last;
        uint64_t mass = 0;
        each([&](uint64_t pl, auto w) { if (pl >= last) mass += w(); });
        total = group_sum_u64<NT>(mass, s.sum);
        base = 0;
    }
    const uint64_t cut = narrow_cut<NT>(s, p_target(p.p, total) - base, each);
    return cut > last ? cut : last;
}

// Index of u's place in a running sum up to `total`.
__device__ __forceinline__ uint64_t drawn_mass(float u, uint64_t total) {
    const double ud = u > 0.0f ? fmin((double)u, 1.0) : 0.0;  // (NaN: 0)
    const uint64_t d = (uint64_t)(ud * (double)total);
    return total && d >= total ? total - 1 : d;
}

// The element at which the running sum of w, in index order, exceeds `draw`: element
// PER tid + j has logit l[j] and weight w[j] in thread tid.  s.token = its number or -1,
// s.logit = its logit; visible after the call.
template <int NT, int PER>
__device__ __forceinline__ void find_drawn(Draw& s, const float (&l)[PER], const uint64_t (&w)[PER],
                                           uint64_t draw) {
    constexpr int NW = NT / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += w[j];
    const uint64_t inc = wave_scan_u64(sum);
    __syncthreads();  // s.sum may still be read
    if (lane == 63) s.sum[wave] = inc;
    if (tid == 0) {
        s.token = -1;
        s.logit = -INFINITY;
    }
    __syncthreads();
    uint64_t run = inc - sum;
#pragma unroll
    for (int v = 0; v < NW; ++v) run += v < wave ? s.sum[v] : 0;
    if (run <= draw && run + sum > draw) {  // one thread
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (run <= draw && run + w[j] > draw) {
                s.token = PER * tid + j;
                s.logit = l[j];
            }
            run += w[j];
        }
    }
    __syncthreads();
}

// The chosen token's outputs; x is its depth (it has a weight, so x < kRange), and total
// the sum of the kept weights, 0 in a row without a live logit.
template <int NT>
__device__ __forceinline__ void write_token(const SampleArgs& a, int b, int token, double x, uint64_t total) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        a.token[b] = token;
        if (a.prob) a.prob[b] = total ? (float)(exp_in(x) / (double)total) : 0.0f;
    }
    if (!a.x_next) return;
    const int d = a.d;
    const size_t r = (size_t)token;
    for (int wd = tid; wd < d / 8; wd += NT) {
        const uint32_t code = a.embed.q[r * (size_t)(d / 8) + wd];
        const size_t g = r * (size_t)(d / kGroup) + wd / 8;
        *(bf16x8*)(a.x_next + (size_t)b * d + 8 * (size_t)wd) =
            dequant8(code, dq_scale(a.embed.scale[g]), bf16_to_f32(a.embed.bias[g]));
    }
}

// R: aligned 16-byte pieces of a chunk per thread, chunk / (4 NT) + 1 (a row that does not
// start on a piece has one more).
template <int NT, int R>
__global__ __launch_bounds__(NT) void sample_pick_kernel(const SampleArgs a) {
    constexpr int NW = NT / 64;
    constexpr int LPT = kList / NT;  // list entries per thread
    static_assert(kMaxChunks <= NT, "one chunk a thread");
    __shared__ Draw s;
    __shared__ unsigned long long s_chunk[kMaxChunks];
    __shared__ uint64_t s_seg[R * NW];
    __shared__ int s_at;
    __shared__ uint64_t s_before;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // everything that the earlier kernels left, in one round trip (entries past the
    // list's end are read, inside the workspace, and not used)
    const SampleRow p = a.row[b];
    const uint32_t n = a.list_n[b];
    const SampleState st = a.state[b];
    const int cc = tid < a.n_chunks ? tid : 0;
    const float pm = a.part_max[(size_t)b * a.n_chunks + cc];
    const uint64_t cw = a.chunk_w[(size_t)b * a.n_chunks + cc];
    uint64_t lp[LPT], lw[LPT];
#pragma unroll
    for (int j = 0; j < LPT; ++j) lp[j] = a.list[(size_t)b * kList + tid + j * NT];
    const double m = (double)fminf(group_max_f<NT>(pm, s.m), FLT_MAX);
    if (tid < a.n_chunks) s_chunk[tid] = cw;
    const float* row = a.logits + (size_t)b * a.V;
    uint64_t last = 0;  // kept: place >= last
    if (m > -INFINITY && (p.cut_k || p.cut_p)) {
        const bool listed = n <= (uint32_t)kList;
#pragma unroll
        for (int j = 0; j < LPT; ++j) {
            lw[j] = 0;
            if (listed && tid + j * NT < (int)n) lw[j] = weight(place_logit(lp[j]), m, p.inv_t);
        }
        auto each = [&](auto f) {
            if (listed) {
#pragma unroll
                for (int j = 0; j < LPT; ++j)
                    if (lw[j]) f(lp[j], [&] { return lw[j]; });
            } else {
                // the whole row, eight logits of a thread in flight
                for (int i0 = tid; i0 < a.V; i0 += 8 * NT) {
                    float l[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) l[q] = row[min(i0 + q * NT, a.V - 1)];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int i = i0 + q * NT;
                        const double x = depth(l[q], m, p.inv_t);
                        if (i < a.V && x < kRange) {
                            const int bin = bin_of(x);
                            if (bin >= st.lo && bin <= st.hi) f(place(l[q], i), [&] { return weight_in(x); });
                        }
                    }
                }
            }
        };
        last = row_cut<NT>(s, p, st.reached, st.before, st.total, n <= (uint32_t)kRank, each);
        __syncthreads();
        each([&](uint64_t pl, auto weight_of) {
            if (pl < last) return;
            const uint64_t w = weight_of();
            if (w >= p.w_min) atomicAdd(&s_chunk[place_index(pl) >> a.chunk_sh], (unsigned long long)w);
        });
    }
    __syncthreads();
    // the chunk that holds the drawn mass
    const uint64_t mine = tid < a.n_chunks ? s_chunk[tid] : 0;
    const uint64_t inc_w = wave_scan_u64(mine);
    if (lane == 63) s.sum[wave] = inc_w;
    if (tid == 0) {
        s_at = -1;
        s.token = 0;
        s.logit = -INFINITY;
    }
    __syncthreads();
    uint64_t run = inc_w - mine, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        run += w < wave ? s.sum[w] : 0;
        total += s.sum[w];
    }
    const uint64_t draw = drawn_mass(p.u, total);
    if (mine && run <= draw && run + mine > draw) {
        s_at = tid;
        s_before = run;
    }
    __syncthreads();
    int token = 0;
    float logit = -INFINITY;
    const int chunk = s_at;
    if (chunk >= 0) {  // (uniform; a row without a live logit has total 0 and token 0)
        const int i0 = chunk << a.chunk_sh;
        const int i1 = min(a.V, i0 + (1 << a.chunk_sh));
        const int64_t o = (int64_t)b * a.V, size = (int64_t)a.B * a.V;
        const int64_t g0 = (o + i0) >> 2, g1 = (o + i1 + 3) >> 2;
        f32x4 l[R];
        uint64_t sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t g = g0 + r * NT + tid;
            l[r] = load_piece(a.logits, g < g1 ? g : g0, size);
        }
        auto kept_weight = [&](float v, int i) {
            const uint64_t w = weight(v, m, p.inv_t);
            return w < p.w_min || place(v, i) < last ? 0 : w;
        };
#pragma unroll
        for (int r = 0; r < R; ++r) {  // sums of 256 neighbouring elements, in index order
            const int64_t g = g0 + r * NT + tid;
            const int base = (int)(4 * g - o);
            sum[r] = 0;
            if (g < g1) {
                mask_piece(l[r], base, i0, i1);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[r] += kept_weight(l[r][j], base + j);
            }
            const uint64_t t = wave_sum_u64(sum[r]);
            if (lane == 0) s_seg[r * NW + wave] = t;
        }
        __syncthreads();
        const uint64_t want = draw - s_before;
        uint64_t before = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {  // (uniform over the wave)
            uint64_t row_before = before;
            for (int v = 0; v < NW; ++v) {
                const uint64_t seg = s_seg[r * NW + v];
                row_before += v < wave ? seg : 0;
                before += seg;
            }
            if (row_before <= want && row_before + s_seg[r * NW + wave] > want) {
                uint64_t at = row_before + wave_scan_u64(sum[r]) - sum[r];
                if (at <= want && at + sum[r] > want) {  // one thread of the work group
                    const int base = (int)(4 * (g0 + r * NT + tid) - o);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t w = kept_weight(l[r][j], base + j);
                        if (at <= want && at + w > want) {
                            s.token = base + j;
                            s.logit = l[r][j];
                        }
                        at += w;
                    }
                }
            }
        }
        __syncthreads();
        token = s.token;
        logit = s.logit;
    }
    write_token<NT>(a, b, token, depth(logit, m, p.inv_t), total);
}

// A short row (V <= NT PER): element PER tid + j in register j of thread tid.  Weights are
// computed where they are used: kept in registers beside the logits they spill.
template <int NT, int PER>
__global__ __launch_bounds__(NT) void sample_row_kernel(const SampleArgs a) {
    __shared__ Draw s;
    const int b = blockIdx.x, tid = threadIdx.x;
    const float* row = a.logits + (size_t)b * a.V;
    float l[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = PER * tid + j;
        l[j] = row[i < a.V ? i : a.V - 1];
    }
    const SampleRow p = row_params(a, b);
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (PER * tid + j >= a.V) l[j] = -INFINITY;
        most = fmaxf(most, l[j]);
    }
    const double m = (double)fminf(group_max_f<NT>(most, s.m), FLT_MAX);
    uint64_t last = 0;
    if (m > -INFINITY && (p.cut_k || p.cut_p)) {
        for (int i = tid; i < kBins; i += NT) s.hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const double x = depth(l[j], m, p.inv_t);
            if (x < kRange)
                atomicAdd((unsigned long long*)&s.hist[bin_of(x)],
                          p.cut_k ? 1ull : (unsigned long long)weight_in(x));
        }
        __syncthreads();
        const Cut cut = find_cut<NT>(s.hist, s.cs, [&](uint64_t total) {
            return p.cut_k ? (uint64_t)p.k : p_target(p.p, total);
        });
        const int hi = min(cut.bin, kBins - 1), lo = p.cut_k ? 0 : hi;
        auto each = [&](auto f) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const double x = depth(l[j], m, p.inv_t);
                if (x < kRange) {
                    const int bin = bin_of(x);
                    if (bin >= lo && bin <= hi) f(place(l[j], PER * tid + j), [&] { return weight_in(x); });
                }
            }
        };
        last = row_cut<NT>(s, p, cut.bin < kBins, cut.before, cut.total, true, each);
    }
    uint64_t w[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        w[j] = weight(l[j], m, p.inv_t);
        if (w[j] < p.w_min || place(l[j], PER * tid + j) < last) w[j] = 0;
        sum += w[j];
    }
    const uint64_t total = group_sum_u64<NT>(sum, s.sum);
    find_drawn<NT, PER>(s, l, w, drawn_mass(p.u, total));
    write_token<NT>(a, b, max(s.token, 0), depth(s.logit, m, p.inv_t), total);
}

}  // namespace

// log2 of the logits per chunk: about 1024 work groups.  (64 rows of 248320: the histogram
// kernel takes 25 us with 970 work groups and 33 with 1984, whose histograms are flushed
// twice as often.)
static_assert((MOE_MAX_VOCAB >> 11) <= kSampleMaxChunks, "chunks of a row");
int sample_chunk_sh(int V, int B) {
    int sh = 11;  // .. 14: V <= 2^20 makes at most 512 chunks of 2048
    auto chunks = [&] { return (V + (1 << sh) - 1) >> sh; };
    while (sh < 14 && (int64_t)B * chunks() > 1024) ++sh;
    return sh;
}

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
    hipError_t e;
    if (a.V <= kSampleRowMax) {
        // 4096 logits: 6.8 us (temperature alone) and 11.5 (top-p) against 12.6 and 18.6 of the
        // four kernels; 16384 with 16 a thread: 17.3 and 28.6 against 12.9 and 19.0
        if (a.V <= 4096) sample_row_kernel<512, 8><<<a.B, 512, 0, s>>>(a);
        else sample_row_kernel<1024, 8><<<a.B, 1024, 0, s>>>(a);
        trace_point(s);
        return hipGetLastError();
    }
    const dim3 grid(a.n_chunks, a.B);
    sample_max_kernel<<<grid, kThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    trace_point(s);
    sample_hist_kernel<<<grid, kThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    trace_point(s);
    sample_gather_kernel<<<grid, kThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    trace_point(s);
    if (a.chunk_sh == 11) sample_pick_kernel<512, 2><<<a.B, 512, 0, s>>>(a);
    else if (a.chunk_sh == 12) sample_pick_kernel<512, 3><<<a.B, 512, 0, s>>>(a);
    else if (a.chunk_sh == 13) sample_pick_kernel<1024, 3><<<a.B, 1024, 0, s>>>(a);
    else sample_pick_kernel<1024, 5><<<a.B, 1024, 0, s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
