// sample.hip -- one token per row of logits: temperature, top-k, top-p, min-p and
// a draw from a given uniform number (moe_sample).
//
// Order of a row's tokens: larger logit first, equal logits by the lower index; all
// three filters keep a prefix of that order.  Weights are
//   w_i = round(2^43 exp(-x_i)),  x_i = (l_max - l_i) / temperature < 30.4
// (0 beyond, where the rounding gives at most 1) as 64-bit integers, so every sum is
// exact (V <= 2^20 weights of at most 2^43) and the same in any order: atomics and
// split sums give the same token every time, and a weight's rounding, 2^-44 of the
// largest, is far below the step of a 24-bit uniform number.
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
// itself.  If the list overflows (thousands of equal logits at the cut), kernel 4
// narrows over the whole row instead.
// Short rows (sample_row_kernel): one work group does all of it with the row in its
// registers.
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kThreads = 256;       // of kernels 1 to 3
constexpr int kPickThreads = 1024;  // of kernel 4 and of the short rows' kernel
constexpr int kPickWaves = kPickThreads / 64;
constexpr int kBins = kSampleBins;
constexpr int kList = kSampleList;
constexpr int kRank = 256;          // tokens ranked against each other at once
constexpr int kMaxChunks = kSampleMaxChunks;
constexpr int kIdxBits = 20;        // MOE_MAX_VOCAB = 2^20
constexpr double kOne = 8796093022208.0;  // 2^43: the weight of the largest logit
constexpr double kRange = 30.4;           // beyond this depth a weight is 0

// One row's parameters.
struct Row {
    double inv_t;      // 1 / temperature
    uint32_t k;        // tokens top-k keeps, 1 .. V
    bool cut_k, cut_p; // top-k / top-p are on
    double p;
    uint64_t w_min;    // min-p: the smallest kept weight, >= 1
};

__device__ __forceinline__ float param(const float* a, float all, int b) { return a ? a[b] : all; }

__device__ __forceinline__ Row row_params(const SampleArgs& a, int b) {
    Row r;
    const float t = param(a.temperature, a.temperature_all, b);
    const bool greedy = !(t > 0.0f);
    r.inv_t = greedy ? 1.0 : 1.0 / (double)t;
    const int k = a.top_k ? a.top_k[b] : a.top_k_all;
    r.k = greedy ? 1u : (k <= 0 || k > a.V) ? (uint32_t)a.V : (uint32_t)k;
    r.cut_k = r.k < (uint32_t)a.V;
    const float p = param(a.top_p, a.top_p_all, b);
    r.cut_p = p < 1.0f && !greedy;
    r.p = p > 0.0f ? (double)p : 0.0;
    float mp = param(a.min_p, a.min_p_all, b);
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

// Depth x of a logit; infinite for a masked logit or a NaN (never NaN itself:
// infinity - infinity is taken out, and 0 * infinity, which the temperature
// infinity gives, counts as out of range below).
__device__ __forceinline__ double depth(float l, float m, double inv_t) {
    if (!(l > -INFINITY)) return INFINITY;
    return l == m ? 0.0 : ((double)m - (double)l) * inv_t;
}

// Bin of a depth below kRange; deeper logits have higher bins.
__device__ __forceinline__ int bin_of(double x) {
    return min(kBins - 1, (int)(x * (kBins / kRange)));
}

// round(2^43 exp(-x)) for 0 <= x < kRange, else 0.  x = n ln 2 - r with |r| <= ln 2 / 2,
// exp(r) by its Taylor series to r^11 / 11! (next term below 2^-47), and the rounding
// by adding 2^52, which leaves the integer in the low bits of the sum.
__device__ __forceinline__ uint64_t weight_at(double x) {
    if (!(x < kRange)) return 0;
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(n, 0.69314718055994529, -x);  // ln 2 in two parts
    r = __builtin_fma(n, 2.3190468138462996e-17, r);
    double e = 1.0 / 39916800.0;
    e = __builtin_fma(e, r, 1.0 / 3628800.0);
    e = __builtin_fma(e, r, 1.0 / 362880.0);
    e = __builtin_fma(e, r, 1.0 / 40320.0);
    e = __builtin_fma(e, r, 1.0 / 5040.0);
    e = __builtin_fma(e, r, 1.0 / 720.0);
    e = __builtin_fma(e, r, 1.0 / 120.0);
    e = __builtin_fma(e, r, 1.0 / 24.0);
    e = __builtin_fma(e, r, 1.0 / 6.0);
    e = __builtin_fma(e, r, 0.5);
    e = __builtin_fma(e, r, 1.0);
    e = __builtin_fma(e, r, 1.0);
    const double v = __builtin_ldexp(e, 43 - (int)n) + 4503599627370496.0;
    return (uint64_t)__double_as_longlong(v) & 0xFFFFFFFFFFFFFull;
}

__device__ __forceinline__ uint64_t weight(float l, float m, double inv_t) {
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

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
    return v;
}

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// Inclusive running sum over the wave's lanes.
__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = __shfl_up(v, o, kWave);
        if (lane >= o) v += y;
    }
    return v;
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

// The row's largest logit from the chunks' (every thread; s: one entry per wave).
template <int NT>
__device__ __forceinline__ float row_max(const SampleArgs& a, int b, float* s) {
    float m = -INFINITY;
    for (int c = threadIdx.x; c < a.n_chunks; c += NT) m = fmaxf(m, a.part_max[(size_t)b * a.n_chunks + c]);
    return group_max_f<NT>(m, s);
}

// Calls f(logit, index) for this thread's elements of row b in [i0, i1).  The logits
// come in aligned 16-byte pieces whatever V is: a piece at an end of the range may hold
// elements outside it, which are passed over, and the piece that would cross the end of
// the whole array is read element by element.
template <int NT, typename F>
__device__ __forceinline__ void each_logit(const SampleArgs& a, int b, int i0, int i1, F f) {
    const int64_t o = (int64_t)b * a.V, total = (int64_t)a.B * a.V;
    const int64_t g1 = (o + i1 + 3) >> 2;
    for (int64_t g0 = ((o + i0) >> 2) + threadIdx.x; g0 < g1; g0 += 4 * NT) {
        f32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // four pieces in flight
            const int64_t g = g0 + u * NT;
            if (g < g1) {
                if (4 * g + 4 <= total) {
                    v[u] = *(const f32x4*)(a.logits + 4 * g);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[u][j] = 4 * g + j < total ? a.logits[4 * g + j] : 0.0f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t g = g0 + u * NT;
            if (g >= g1) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = (int)(4 * g + j - o);
                if (i >= i0 && i < i1) f(v[u][j], i);
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void sample_max_kernel(const SampleArgs a) {
    __shared__ float s[kThreads / 64];
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    // the row's histogram and counter, shared out over its chunks
    for (int i = c * kThreads + tid; i < kBins; i += a.n_chunks * kThreads) a.hist[(size_t)b * kBins + i] = 0;
    if (c == 0 && tid == 0) a.list_n[b] = 0;
    const int i0 = c << a.chunk_sh, i1 = min(a.V, i0 + (1 << a.chunk_sh));
    float m = -INFINITY;
    each_logit<kThreads>(a, b, i0, i1, [&](float l, int) { m = fmaxf(m, l); });  // (NaN is passed over)
    m = group_max_f<kThreads>(m, s);
    if (tid == 0) a.part_max[(size_t)b * a.n_chunks + c] = m;
}

__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const SampleArgs a) {
    __shared__ unsigned long long s_h[kBins];
    __shared__ float s_m[kThreads / 64];
    __shared__ uint64_t s_sum[kThreads / 64];
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const Row p = row_params(a, b);
    const float m = row_max<kThreads>(a, b, s_m);
    const int i0 = c << a.chunk_sh, i1 = min(a.V, i0 + (1 << a.chunk_sh));
    if (!p.cut_k && !p.cut_p) {  // uniform over the work group
        uint64_t sum = 0;
        each_logit<kThreads>(a, b, i0, i1, [&](float l, int) {
            const uint64_t w = weight(l, m, p.inv_t);
            sum += w >= p.w_min ? w : 0;
        });
        sum = group_sum_u64<kThreads>(sum, s_sum);
        if (tid == 0) a.chunk_w[(size_t)b * a.n_chunks + c] = sum;
        return;
    }
    for (int i = tid; i < kBins; i += kThreads) s_h[i] = 0;
    __syncthreads();
    each_logit<kThreads>(a, b, i0, i1, [&](float l, int) {
        const double x = depth(l, m, p.inv_t);
        if (x < kRange) atomicAdd(&s_h[bin_of(x)], p.cut_k ? 1ull : (unsigned long long)weight_at(x));
    });
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
    uint64_t wave[kPickWaves];
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
    const uint64_t inc = wave_scan_u64(sum, lane);
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
    __shared__ unsigned long long s_list[kList];
    __shared__ uint32_t s_n, s_base;
    __shared__ float s_m[kThreads / 64];
    __shared__ uint64_t s_sum[kThreads / 64];
    __shared__ CutScratch s_cut;
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const Row p = row_params(a, b);
    if (!p.cut_k && !p.cut_p) return;  // uniform
    const float m = row_max<kThreads>(a, b, s_m);
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
    const int i0 = c << a.chunk_sh, i1 = min(a.V, i0 + (1 << a.chunk_sh));
    uint64_t sum = 0;
    each_logit<kThreads>(a, b, i0, i1, [&](float l, int i) {
        const double x = depth(l, m, p.inv_t);
        if (!(x < kRange)) return;
        const int bin = bin_of(x);
        if (bin < lo) {
            const uint64_t w = weight_at(x);
            sum += w >= p.w_min ? w : 0;
        } else if (bin <= hi) {
            const uint32_t at = atomicAdd(&s_n, 1u);
            if (at < (uint32_t)kList) s_list[at] = place(l, i);
        }
    });
    sum = group_sum_u64<kThreads>(sum, s_sum);  // (its barriers also complete the list)
    const uint32_t n = s_n;
    if (tid == 0) {
        a.chunk_w[(size_t)b * a.n_chunks + c] = sum;
        s_base = n ? atomicAdd(&a.list_n[b], n) : 0;
    }
    __syncthreads();
    // a list that overflows is not used: list_n says so
    if (n <= (uint32_t)kList && s_base + n <= (uint32_t)kList)
        for (uint32_t i = tid; i < n; i += kThreads) a.list[(size_t)b * kList + s_base + i] = s_list[i];
}

// Shared memory of the work group that makes a row's cut and draw.
struct Draw {
    uint64_t hist[kBins];
    uint64_t rank_p[kRank], rank_q[kRank];
    unsigned long long lo, hi, cut;
    uint32_t n;
    CutScratch cs;
    uint64_t seg[16 * kPickWaves];  // sums of 64 neighbouring elements, in index order
    uint64_t sum[kPickWaves];
    float m[kPickWaves];
    int token;
    uint64_t wt;
};

// The last kept token of a region: the first, in the row's order, at which the running
// sum of a quantity reaches the target (some token does).  each(f) calls f(place,
// quantity) for this thread's tokens of the region.  Tokens are narrowed down by their
// place, a factor of 2048 a time, until kRank of them are left, which are ranked by
// comparing each with each.  Returns the token's place.
template <typename Each>
__device__ __forceinline__ uint64_t narrow_cut(Draw& s, uint64_t target, Each each) {
    const int tid = threadIdx.x, lane = tid & 63;
    uint64_t lo = 0, hi = ~0ull;
    for (bool first = true;; first = false) {
        __syncthreads();
        if (tid == 0) {
            s.n = 0;
            s.cut = 0;  // (not reached: everything is kept)
            s.lo = ~0ull;
            s.hi = 0;
        }
        __syncthreads();
        each([&](uint64_t p, uint64_t q) {
            if (p >= lo && p <= hi && s.n <= (uint32_t)kRank) {
                const uint32_t at = atomicAdd(&s.n, 1u);
                if (at < (uint32_t)kRank) {
                    s.rank_p[at] = p;
                    s.rank_q[at] = q;
                }
            }
        });
        __syncthreads();
        const int n = (int)min(s.n, (uint32_t)kRank + 1);
        if (n <= kRank) {
            // four threads per token, each over a quarter of the others
            const int i = tid >> 2;
            if (i < n) {
                const uint64_t p = s.rank_p[i];
                uint64_t run = 0;
                for (int j = tid & 3; j < n; j += 4) run += s.rank_p[j] > p ? s.rank_q[j] : 0;
                run += __shfl_xor(run, 1, kWave);
                run += __shfl_xor(run, 2, kWave);
                if (run < target && run + s.rank_q[i] >= target) s.cut = p;
            }
            __syncthreads();
            return s.cut;
        }
        if (first) {
            uint64_t l = ~0ull, h = 0;
            each([&](uint64_t p, uint64_t) {
                l = p < l ? p : l;
                h = p > h ? p : h;
            });
            if (h >= l) {
                atomicMin(&s.lo, l);
                atomicMax(&s.hi, h);
            }
            __syncthreads();
            lo = s.lo;
            hi = s.hi;
        }
        const int bits = 64 - __builtin_clzll(hi - lo);  // (more than kRank places: hi > lo)
        const int shift = bits > 11 ? bits - 11 : 0;
        for (int i = tid; i < kBins; i += kPickThreads) s.hist[i] = 0;
        __syncthreads();
        each([&](uint64_t p, uint64_t q) {
            if (p >= lo && p <= hi)
                atomicAdd((unsigned long long*)&s.hist[(int)((hi - p) >> shift)], (unsigned long long)q);
        });
        __syncthreads();
        const Cut c = find_cut<kPickThreads>(s.hist, s.cs, [&](uint64_t) { return target; });
        if (c.bin >= kBins) return 0;
        target -= c.before;
        hi -= (uint64_t)c.bin << shift;
        if (shift == 0) return hi;
        const uint64_t bottom = hi - ((1ull << shift) - 1);
        lo = bottom > lo ? bottom : lo;
    }
    (void)lane;
}

// The cut of a row whose region's tokens each(f) visits as f(place, weight): top-k (if
// its target lies in the region), then top-p.  base: mass before the region, total: the
// mass top-p refers to without top-k.
template <typename Each>
__device__ __forceinline__ uint64_t row_cut(Draw& s, const Row& p, bool k_reached, uint64_t base,
                                            uint64_t total, Each each) {
    uint64_t last = 0;
    if (p.cut_k) {
        if (k_reached)
            last = narrow_cut(s, p.k, [&](auto f) { each([&](uint64_t pl, uint64_t) { f(pl, 1ull); }); });
        if (!p.cut_p) return last;
        uint64_t mass = 0;
        each([&](uint64_t pl, uint64_t w) { mass += pl >= last ? w : 0; });
        total = group_sum_u64<kPickThreads>(mass, s.sum);
        base = 0;
    }
    const uint64_t cut = narrow_cut(s, p_target(p.p, total) - base, each);
    return cut > last ? cut : last;
}

// Index of u's place in a running sum up to `total`.
__device__ __forceinline__ uint64_t drawn_mass(float u, uint64_t total) {
    const double ud = u > 0.0f ? fmin((double)u, 1.0) : 0.0;  // (NaN: 0)
    const uint64_t d = (uint64_t)(ud * (double)total);
    return total && d >= total ? total - 1 : d;
}

// The element at which the running sum of w, in index order, exceeds `draw`: element
// 1024 j + tid has weight w[j] in thread tid.  s.token = its number or -1, s.wt = its
// weight; visible after the call.  total: the sum of all w.
template <int PER>
__device__ __forceinline__ void find_drawn(Draw& s, const uint64_t (&w)[PER], uint64_t draw) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const uint64_t t = wave_sum_u64(w[j]);
        if (lane == 0) s.seg[j * kPickWaves + wave] = t;
    }
    if (tid == 0) {
        s.token = -1;
        s.wt = 0;
    }
    __syncthreads();
    // every wave finds the segment; the one that holds it looks through its lanes
    constexpr int SEG = PER * kPickWaves, EACH = (SEG + 63) / 64;
    uint64_t v[EACH], sum = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        v[e] = lane * EACH + e < SEG ? s.seg[lane * EACH + e] : 0;
        sum += v[e];
    }
    uint64_t run = wave_scan_u64(sum, lane) - sum;
    int seg = -1;
    uint64_t before = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        if (run <= draw && run + v[e] > draw) {
            seg = lane * EACH + e;
            before = run;
        }
        run += v[e];
    }
    const uint64_t who = __ballot(seg >= 0);
    if (who) {  // uniform
        const int from = (int)__builtin_ctzll(who);
        seg = __shfl(seg, from, kWave);
        before = __shfl(before, from, kWave);
        if (seg % kPickWaves == wave) {
            uint64_t mine = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) mine = seg / kPickWaves == j ? w[j] : mine;
            const uint64_t inc = before + wave_scan_u64(mine, lane);
            if (mine && inc > draw && inc - mine <= draw) {
                s.token = seg * 64 + lane;
                s.wt = mine;
            }
        }
    }
    __syncthreads();
}

// The chosen token's outputs.
__device__ __forceinline__ void write_token(const SampleArgs& a, int b, int token, uint64_t wt,
                                            uint64_t total) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        a.token[b] = token;
        if (a.prob) a.prob[b] = total ? (float)((double)wt / (double)total) : 0.0f;
    }
    if (!a.x_next) return;
    const int d = a.d;
    const size_t r = (size_t)token;
    for (int wd = tid; wd < d / 8; wd += kPickThreads) {
        const uint32_t code = a.embed.q[r * (size_t)(d / 8) + wd];
        const size_t g = r * (size_t)(d / kGroup) + wd / 8;
        *(bf16x8*)(a.x_next + (size_t)b * d + 8 * (size_t)wd) =
            dequant8(code, dq_scale(a.embed.scale[g]), bf16_to_f32(a.embed.bias[g]));
    }
}

// PER: elements of a chunk per thread, chunk / 1024.
template <int PER>
__global__ __launch_bounds__(kPickThreads) void sample_pick_kernel(const SampleArgs a) {
    constexpr int LPT = kList / kPickThreads;  // list entries per thread
    __shared__ Draw s;
    __shared__ unsigned long long s_chunk[kMaxChunks];
    __shared__ int s_at;
    __shared__ uint64_t s_before;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Row p = row_params(a, b);
    const uint32_t n = a.list_n[b];
    const float u = a.u[b];
    const float m = row_max<kPickThreads>(a, b, s.m);
    for (int c = tid; c < a.n_chunks; c += kPickThreads) s_chunk[c] = a.chunk_w[(size_t)b * a.n_chunks + c];
    const float* row = a.logits + (size_t)b * a.V;
    uint64_t last = 0;  // kept: place >= last
    if (m > -INFINITY && (p.cut_k || p.cut_p)) {
        const SampleState st = a.state[b];
        const bool listed = n <= (uint32_t)kList;
        uint64_t lp[LPT], lw[LPT];
#pragma unroll
        for (int j = 0; j < LPT; ++j) {
            const uint32_t i = tid + j * kPickThreads;
            const bool live = listed && i < n;
            lp[j] = live ? a.list[(size_t)b * kList + i] : 0;
            lw[j] = live ? weight(place_logit(lp[j]), m, p.inv_t) : 0;
        }
        auto each = [&](auto f) {
            if (listed) {
#pragma unroll
                for (int j = 0; j < LPT; ++j)
                    if (lw[j]) f(lp[j], lw[j]);
            } else {
                for (int i = tid; i < a.V; i += kPickThreads) {
                    const double x = depth(row[i], m, p.inv_t);
                    if (!(x < kRange)) continue;
                    const int bin = bin_of(x);
                    if (bin >= st.lo && bin <= st.hi) f(place(row[i], i), weight_at(x));
                }
            }
        };
        last = row_cut(s, p, st.reached, st.before, st.total, each);
        __syncthreads();
        each([&](uint64_t pl, uint64_t w) {
            if (pl >= last && w >= p.w_min)
                atomicAdd(&s_chunk[place_index(pl) >> a.chunk_sh], (unsigned long long)w);
        });
    }
    __syncthreads();
    // the chunk that holds the drawn mass (kMaxChunks <= 1024: one a thread)
    const uint64_t mine = tid < a.n_chunks ? s_chunk[tid] : 0;
    const uint64_t inc_w = wave_scan_u64(mine, lane);
    if (lane == 63) s.sum[wave] = inc_w;
    if (tid == 0) s_at = -1;
    __syncthreads();
    uint64_t run = inc_w - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kPickWaves; ++w) {
        run += w < wave ? s.sum[w] : 0;
        total += s.sum[w];
    }
    const uint64_t draw = drawn_mass(u, total);
    if (mine && run <= draw && run + mine > draw) {
        s_at = tid;
        s_before = run;
    }
    __syncthreads();
    int token = 0;
    uint64_t wt = 0;
    const int chunk = s_at;
    if (chunk >= 0) {  // (uniform; a row without a live logit has total 0 and token 0)
        const int i0 = chunk << a.chunk_sh;
        uint64_t w[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = i0 + j * kPickThreads + tid;
            w[j] = 0;
            if (i < a.V) {
                const float l = row[i];
                w[j] = weight(l, m, p.inv_t);
                if (w[j] < p.w_min || place(l, i) < last) w[j] = 0;
            }
        }
        find_drawn<PER>(s, w, draw - s_before);
        token = s.token >= 0 ? i0 + s.token : 0;
        wt = s.wt;
    }
    write_token(a, b, token, wt, total);
}

// A short row (V <= 1024 PER): element 1024 j + tid in register j of thread tid.
template <int PER>
__global__ __launch_bounds__(kPickThreads) void sample_row_kernel(const SampleArgs a) {
    __shared__ Draw s;
    const int b = blockIdx.x, tid = threadIdx.x;
    const Row p = row_params(a, b);
    const float u = a.u[b];
    const float* row = a.logits + (size_t)b * a.V;
    float l[PER];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * kPickThreads + tid;
        l[j] = i < a.V ? row[i] : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) m = fmaxf(m, l[j]);
    m = group_max_f<kPickThreads>(m, s.m);
    uint64_t w[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) w[j] = weight(l[j], m, p.inv_t);
    uint64_t last = 0;
    if (m > -INFINITY && (p.cut_k || p.cut_p)) {
        for (int i = tid; i < kBins; i += kPickThreads) s.hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (w[j])
                atomicAdd((unsigned long long*)&s.hist[bin_of(depth(l[j], m, p.inv_t))],
                          p.cut_k ? 1ull : (unsigned long long)w[j]);
        __syncthreads();
        const Cut cut = find_cut<kPickThreads>(s.hist, s.cs, [&](uint64_t total) {
            return p.cut_k ? (uint64_t)p.k : p_target(p.p, total);
        });
        const int hi = min(cut.bin, kBins - 1), lo = p.cut_k ? 0 : hi;
        auto each = [&](auto f) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (w[j]) {
                    const int bin = bin_of(depth(l[j], m, p.inv_t));
                    if (bin >= lo && bin <= hi) f(place(l[j], j * kPickThreads + tid), w[j]);
                }
        };
        last = row_cut(s, p, cut.bin < kBins, cut.before, cut.total, each);
    }
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (w[j] < p.w_min || place(l[j], j * kPickThreads + tid) < last) w[j] = 0;
        sum += w[j];
    }
    const uint64_t total = group_sum_u64<kPickThreads>(sum, s.sum);
    find_drawn<PER>(s, w, drawn_mass(u, total));
    write_token(a, b, max(s.token, 0), s.wt, total);
}

}  // namespace

// log2 of the logits per chunk: enough chunks for the chip, at most kSampleMaxChunks
// a row.
int sample_chunk_sh(int V, int B) {
    int sh = 11;
    auto chunks = [&] { return (V + (1 << sh) - 1) >> sh; };
    while (chunks() > kSampleMaxChunks || (sh < 14 && (int64_t)B * chunks() > 2048)) ++sh;
    return sh;
}

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
    hipError_t e;
    if (a.V <= kSampleRowMax) {
        if (a.V <= 4 * kPickThreads) sample_row_kernel<4><<<a.B, kPickThreads, 0, s>>>(a);
        else sample_row_kernel<16><<<a.B, kPickThreads, 0, s>>>(a);
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
    if (a.chunk_sh == 11) sample_pick_kernel<2><<<a.B, kPickThreads, 0, s>>>(a);
    else if (a.chunk_sh == 12) sample_pick_kernel<4><<<a.B, kPickThreads, 0, s>>>(a);
    else if (a.chunk_sh == 13) sample_pick_kernel<8><<<a.B, kPickThreads, 0, s>>>(a);
    else sample_pick_kernel<16><<<a.B, kPickThreads, 0, s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
