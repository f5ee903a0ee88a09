// sample.hip -- one token per row of logits: temperature, top-k, top-p, min-p and
// a draw from a given uniform number (moe_sample).
//
// Order of a row's tokens: larger logit first, equal logits by the lower index; all
// three filters keep a prefix of that order.  Weights are
//   w_i = round(2^43 exp((l_i - l_max) / temperature))
// as 64-bit integers, so every sum is exact (V <= 2^20 weights of at most 2^43) and
// the same in any order: atomics and split sums give the same token every time, and
// a weight's rounding, 2^-44 of the largest, is far below the step of a 24-bit
// uniform number.
//
// The draw runs over the kept tokens in index order, so nothing is ever sorted: all
// that is needed of the order is its cut, the last kept token.  Four kernels, each
// over B x C chunks of the logits but the last:
//   1. sample_max_kernel     largest logit of every chunk; clears the row's histogram
//   2. sample_hist_kernel    count and mass per bin of (l_max - l) / temperature
//                            (2048 bins over the range with nonzero weights)
//   3. sample_gather_kernel  the bin the cut falls into; its tokens into the row's
//                            list, and each chunk's mass above that bin
//   4. sample_pick_kernel    one work group per row: the exact cut by narrowing a
//                            (logit, index) interval over the list, the chunk that
//                            holds the drawn mass, the token in it, its embedding row
// A row without top-k and top-p needs no cut: kernel 2 writes the chunks' masses
// itself.  If more tokens share the cut's bin than the list holds (thousands of equal
// logits), kernel 4 narrows over the whole row instead.
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kThreads = 256;       // of kernels 1 to 3
constexpr int kPickThreads = 1024;  // of kernel 4
constexpr int kBins = kSampleBins;
constexpr int kList = kSampleList;
constexpr int kMaxChunks = kSampleMaxChunks;
constexpr int kIdxBits = 20;        // MOE_MAX_VOCAB = 2^20
constexpr double kOne = 8796093022208.0;  // 2^43: the weight of the largest logit
constexpr double kRange = 31.0;           // exp(-31) rounds to weight 0

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

// (l_max - l) / temperature of a live logit: 0 .. infinity, never NaN.
__device__ __forceinline__ double depth(float l, float m, double inv_t) {
    return l == m ? 0.0 : ((double)m - (double)l) * inv_t;
}

__device__ __forceinline__ uint64_t weight(float l, float m, double inv_t) {
    if (!(l > -INFINITY)) return 0;  // masked, or NaN
    const double x = depth(l, m, inv_t);
    if (!(x < kRange)) return 0;
    return (uint64_t)(exp(-x) * kOne + 0.5);
}

// Bin of a logit with a nonzero weight; deeper logits have higher bins.
__device__ __forceinline__ int bin_of(float l, float m, double inv_t) {
    return min(kBins - 1, (int)(depth(l, m, inv_t) * (kBins / kRange)));
}

// A token's place in the row's order as one number: larger is earlier.
__device__ __forceinline__ uint64_t place(float l, int i) {
    return ((uint64_t)logit_key(l) << kIdxBits) | (uint32_t)((1 << kIdxBits) - 1 - i);
}

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

// The row's largest logit from the chunks' (every thread; s: one entry per wave).
template <int NT>
__device__ __forceinline__ float row_max(const SampleArgs& a, int b, float* s) {
    float m = -INFINITY;
    for (int c = threadIdx.x; c < a.n_chunks; c += NT) m = fmaxf(m, a.part_max[(size_t)b * a.n_chunks + c]);
    m = wave_max_f(m);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
    __syncthreads();
    m = s[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, s[w]);
    return m;
}

__global__ __launch_bounds__(kThreads) void sample_max_kernel(const SampleArgs a) {
    __shared__ float s[kThreads / 64];
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    // the row's histogram and counters, shared out over its chunks
    for (int i = c * kThreads + tid; i < kBins; i += a.n_chunks * kThreads) {
        a.hist_n[(size_t)b * kBins + i] = 0;
        a.hist_w[(size_t)b * kBins + i] = 0;
    }
    if (c == 0 && tid == 0) a.list_n[b] = 0;
    const float* row = a.logits + (size_t)b * a.V;
    const int i0 = c * a.chunk, i1 = min(a.V, i0 + a.chunk);
    float m = -INFINITY;
    for (int i = i0 + tid; i < i1; i += kThreads) m = fmaxf(m, row[i]);  // (NaN is passed over)
    m = wave_max_f(m);
    if ((tid & 63) == 0) s[tid >> 6] = m;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) m = fmaxf(m, s[w]);
        a.part_max[(size_t)b * a.n_chunks + c] = m;
    }
}

__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const SampleArgs a) {
    __shared__ uint32_t s_n[kBins];
    __shared__ unsigned long long s_w[kBins];
    __shared__ float s_m[kThreads / 64];
    __shared__ uint64_t s_sum[kThreads / 64];
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const Row p = row_params(a, b);
    const float m = row_max<kThreads>(a, b, s_m);
    const float* row = a.logits + (size_t)b * a.V;
    const int i0 = c * a.chunk, i1 = min(a.V, i0 + a.chunk);
    if (!p.cut_k && !p.cut_p) {  // uniform over the work group
        uint64_t sum = 0;
        for (int i = i0 + tid; i < i1; i += kThreads) {
            const uint64_t w = weight(row[i], m, p.inv_t);
            sum += w >= p.w_min ? w : 0;
        }
        sum = group_sum_u64<kThreads>(sum, s_sum);
        if (tid == 0) a.chunk_w[(size_t)b * a.n_chunks + c] = sum;
        return;
    }
    for (int i = tid; i < kBins; i += kThreads) {
        s_n[i] = 0;
        s_w[i] = 0;
    }
    __syncthreads();
    for (int i = i0 + tid; i < i1; i += kThreads) {
        const float l = row[i];
        const uint64_t w = weight(l, m, p.inv_t);
        if (w) {
            const int bin = bin_of(l, m, p.inv_t);
            atomicAdd(&s_n[bin], 1u);
            atomicAdd(&s_w[bin], (unsigned long long)w);
        }
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads)
        if (s_n[i]) {
            atomicAdd(&a.hist_n[(size_t)b * kBins + i], s_n[i]);
            atomicAdd((unsigned long long*)&a.hist_w[(size_t)b * kBins + i], s_w[i]);
        }
}

// First bin of NT * PER at which the running count reaches n or the running mass
// reaches w, with what lies before it (count, mass); bin = NT * PER if none.  Called by
// all NT threads; n_of / w_of give a bin's values.
struct Cut {
    int bin;
    uint32_t n;      // tokens before the bin
    uint64_t w;      // their mass
    uint32_t here;   // tokens in it
};

template <int NT, int PER>
__device__ __forceinline__ Cut find_cut(const uint32_t* cn, const uint64_t* cw, uint32_t n, uint64_t w,
                                        uint32_t* s_n, uint64_t* s_w, Cut* s_cut) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t bn[PER], tn = 0;
    uint64_t bw[PER], tw = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        bn[j] = cn[tid * PER + j];
        bw[j] = cw[tid * PER + j];
        tn += bn[j];
        tw += bw[j];
    }
    uint32_t in = tn;
    uint64_t iw = tw;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t x = __shfl_up(in, o, kWave);
        const uint64_t y = __shfl_up(iw, o, kWave);
        if (lane >= o) {
            in += x;
            iw += y;
        }
    }
    __syncthreads();  // the scratch may still be read from the previous use
    if (lane == 63) {
        s_n[wave] = in;
        s_w[wave] = iw;
    }
    if (tid == 0) *s_cut = Cut{NT * PER, 0, 0, 0};
    __syncthreads();
    uint32_t an = in - tn;
    uint64_t aw = iw - tw;
    for (int v = 0; v < wave; ++v) {
        an += s_n[v];
        aw += s_w[v];
    }
    // exactly one thread sees the first crossing
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const bool before = an >= n || aw >= w;
        const bool after = an + bn[j] >= n || aw + bw[j] >= w;
        if (!before && after) *s_cut = Cut{tid * PER + j, an, aw, bn[j]};
        an += bn[j];
        aw += bw[j];
    }
    __syncthreads();
    return *s_cut;
}

// Mass that top-p has to reach: at least 1, so that the first token is kept.
__device__ __forceinline__ uint64_t p_target(double p, uint64_t total) {
    const double t = ceil(p * (double)total);
    return t < 1.0 ? 1ull : (uint64_t)t;
}

__global__ __launch_bounds__(kThreads) void sample_gather_kernel(const SampleArgs a) {
    __shared__ float s_m[kThreads / 64];
    __shared__ uint32_t s_n[kThreads / 64];
    __shared__ uint64_t s_w[kThreads / 64];
    __shared__ Cut s_cut;
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const Row p = row_params(a, b);
    if (!p.cut_k && !p.cut_p) return;  // uniform
    const float m = row_max<kThreads>(a, b, s_m);
    const uint32_t* hn = a.hist_n + (size_t)b * kBins;
    const uint64_t* hw = a.hist_w + (size_t)b * kBins;
    uint64_t mine = 0;
    for (int i = tid; i < kBins; i += kThreads) mine += hw[i];
    const uint64_t total = group_sum_u64<kThreads>(mine, s_w);
    // the bin of the last token that top-k keeps, or (top-p alone) of the one that
    // reaches its mass; with both, top-p's mass is a share of what top-k keeps, so all
    // bins up to top-k's go into the list
    const uint64_t none = ~0ull;
    const Cut cut = find_cut<kThreads, kBins / kThreads>(hn, hw, p.cut_k ? p.k : 0xFFFFFFFFu,
                                                         p.cut_k ? none : p_target(p.p, total), s_n, s_w,
                                                         &s_cut);
    SampleState st;
    if (p.cut_k && cut.bin < kBins) {
        st.lo = 0;
        st.hi = cut.bin;
        st.n = cut.n + cut.here;
        st.base_n = 0;
        st.base_w = 0;
    } else if (!p.cut_k) {  // top-p alone; total >= its target, so there is a bin
        st.lo = st.hi = min(cut.bin, kBins - 1);
        st.n = cut.here;
        st.base_n = cut.n;
        st.base_w = cut.w;
    } else if (p.cut_p) {  // top-k keeps every token with a weight: top-p alone again
        const Cut cp = find_cut<kThreads, kBins / kThreads>(hn, hw, 0xFFFFFFFFu, p_target(p.p, total), s_n,
                                                            s_w, &s_cut);
        st.lo = st.hi = min(cp.bin, kBins - 1);
        st.n = cp.here;
        st.base_n = cp.n;
        st.base_w = cp.w;
    } else {  // nothing is cut
        st.lo = st.hi = kBins;
        st.n = st.base_n = 0;
        st.base_w = 0;
    }
    st.total = total;
    st.k_on = p.cut_k && cut.bin < kBins;
    if (c == 0 && tid == 0) a.state[b] = st;
    const bool listed = st.n <= (uint32_t)kList;
    const float* row = a.logits + (size_t)b * a.V;
    const int i0 = c * a.chunk, i1 = min(a.V, i0 + a.chunk);
    uint64_t sum = 0;
    for (int i = i0 + tid; i < i1; i += kThreads) {
        const float l = row[i];
        const uint64_t w = weight(l, m, p.inv_t);
        if (!w) continue;
        const int bin = bin_of(l, m, p.inv_t);
        if (bin < st.lo) {
            sum += w >= p.w_min ? w : 0;
        } else if (bin <= st.hi && listed) {
            // at most st.n <= kList tokens of the row get here
            const uint32_t at = atomicAdd(&a.list_n[b], 1u);
            if (at < (uint32_t)kList) {
                a.list_p[(size_t)b * kList + at] = place(l, i);
                a.list_w[(size_t)b * kList + at] = w;
            }
        }
    }
    sum = group_sum_u64<kThreads>(sum, s_w);
    if (tid == 0) a.chunk_w[(size_t)b * a.n_chunks + c] = sum;
}

// Shared memory of the narrowing.
struct Narrow {
    uint32_t n[kBins];
    unsigned long long w[kBins];
    unsigned long long lo, hi;
    uint32_t sn[kPickThreads / 64];
    uint64_t sw[kPickThreads / 64];
    Cut cut;
};

// The last kept token of a region: the first one, in the row's order, at which the
// running count reaches n or the running mass reaches w (some token does).  each(f)
// calls f(place, weight) for this thread's tokens of the region.  Returns its place;
// *mass is the region's mass up to and including it.
template <typename Each>
__device__ __forceinline__ uint64_t narrow_cut(Narrow& s, uint32_t n, uint64_t w, uint64_t* mass,
                                               Each each) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) {
        s.lo = ~0ull;
        s.hi = 0;
    }
    __syncthreads();
    uint64_t lo = ~0ull, hi = 0;
    each([&](uint64_t p, uint64_t) {
        lo = p < lo ? p : lo;
        hi = p > hi ? p : hi;
    });
    if (hi >= lo) {
        atomicMin(&s.lo, lo);
        atomicMax(&s.hi, hi);
    }
    __syncthreads();
    lo = s.lo;
    hi = s.hi;
    uint64_t above = 0;  // mass before the interval
    for (;;) {  // [lo, hi] shrinks by a factor of 2048 each time, from at most 2^52
        const uint64_t span = hi - lo;
        const int bits = span ? 64 - __builtin_clzll(span) : 0;
        const int shift = bits > 11 ? bits - 11 : 0;
        for (int i = tid; i < kBins; i += kPickThreads) {
            s.n[i] = 0;
            s.w[i] = 0;
        }
        __syncthreads();
        each([&](uint64_t p, uint64_t wt) {
            if (p >= lo && p <= hi) {
                const int i = (int)((hi - p) >> shift);
                atomicAdd(&s.n[i], 1u);
                atomicAdd(&s.w[i], (unsigned long long)wt);
            }
        });
        __syncthreads();
        const Cut c = find_cut<kPickThreads, kBins / kPickThreads>(s.n, (const uint64_t*)s.w, n, w, s.sn,
                                                                   s.sw, &s.cut);
        if (c.bin >= kBins) {  // not reached: everything is kept
            *mass = above;
            return lo;
        }
        n -= c.n;
        w -= c.w;
        above += c.w;
        hi -= (uint64_t)c.bin << shift;
        if (shift == 0) {
            *mass = above + s.w[c.bin];
            return hi;
        }
        const uint64_t bottom = hi - ((1ull << shift) - 1);
        lo = bottom > lo ? bottom : lo;
        __syncthreads();
    }
}

__global__ __launch_bounds__(kPickThreads) void sample_pick_kernel(const SampleArgs a) {
    __shared__ Narrow s;
    __shared__ unsigned long long s_chunk[kMaxChunks];
    __shared__ float s_m[kPickThreads / 64];
    __shared__ uint64_t s_sum[kPickThreads / 64];
    __shared__ int s_at;
    __shared__ unsigned long long s_before, s_wt;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Row p = row_params(a, b);
    const float m = row_max<kPickThreads>(a, b, s_m);
    const float* row = a.logits + (size_t)b * a.V;
    for (int c = tid; c < a.n_chunks; c += kPickThreads) s_chunk[c] = a.chunk_w[(size_t)b * a.n_chunks + c];
    uint64_t last = 0;  // kept: place >= last
    if (m > -INFINITY && (p.cut_k || p.cut_p)) {
        const SampleState st = a.state[b];
        if (st.lo < kBins) {
            const bool listed = st.n <= (uint32_t)kList;
            auto each = [&](auto f) {
                if (listed) {
                    for (uint32_t i = tid; i < st.n; i += kPickThreads)
                        f((uint64_t)a.list_p[(size_t)b * kList + i], (uint64_t)a.list_w[(size_t)b * kList + i]);
                } else {
                    for (int i = tid; i < a.V; i += kPickThreads) {
                        const float l = row[i];
                        const uint64_t w = weight(l, m, p.inv_t);
                        if (!w) continue;
                        const int bin = bin_of(l, m, p.inv_t);
                        if (bin >= st.lo && bin <= st.hi) f(place(l, i), w);
                    }
                }
            };
            const uint64_t none = ~0ull;
            uint64_t mass = 0;
            if (st.k_on) {
                last = narrow_cut(s, p.k, none, &mass, each);
                if (p.cut_p) last = narrow_cut(s, p.k, p_target(p.p, mass), &mass, each);
            } else {
                last = narrow_cut(s, 0xFFFFFFFFu, p_target(p.p, st.total) - st.base_w, &mass, each);
            }
            __syncthreads();
            each([&](uint64_t pl, uint64_t w) {
                if (pl >= last && w >= p.w_min) {
                    const int i = (1 << kIdxBits) - 1 - (int)(pl & ((1 << kIdxBits) - 1));
                    atomicAdd(&s_chunk[i / a.chunk], (unsigned long long)w);
                }
            });
        }
    }
    __syncthreads();
    // the chunk that holds the drawn mass (a work group of 1024 threads covers
    // kMaxChunks chunks, one a thread)
    const uint64_t mine = tid < a.n_chunks ? s_chunk[tid] : 0;
    const uint64_t total = group_sum_u64<kPickThreads>(mine, s_sum);
    if (tid == 0) {
        s_at = -1;
        s_before = 0;
        s_wt = 0;
    }
    const float u = a.u[b];
    const double ud = u > 0.0f ? fmin((double)u, 1.0) : 0.0;
    uint64_t draw = (uint64_t)(ud * (double)total);
    if (total && draw >= total) draw = total - 1;
    auto scan = [&](uint64_t v) {  // inclusive running sum over the work group
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint64_t y = __shfl_up(v, o, kWave);
            if (lane >= o) v += y;
        }
        __syncthreads();
        if (lane == 63) s_sum[wave] = v;
        __syncthreads();
        for (int x = 0; x < wave; ++x) v += s_sum[x];
        return v;
    };
    {
        const uint64_t inc = scan(mine);
        if (mine && inc > draw && inc - mine <= draw) {
            s_at = tid;
            s_before = inc - mine;
        }
    }
    __syncthreads();
    int token = 0;
    const int chunk = s_at;
    if (chunk >= 0) {  // (uniform; a row without a live logit has total 0 and token 0)
        // the token in the chunk, in index order
        uint64_t before = s_before;
        const int i0 = chunk * a.chunk, i1 = min(a.V, i0 + a.chunk);
        __syncthreads();
        if (tid == 0) s_at = -1;
        __syncthreads();
        for (int base = i0; base < i1; base += kPickThreads) {  // uniform
            const int i = base + tid;
            uint64_t w = 0;
            if (i < i1) {
                const float l = row[i];
                w = weight(l, m, p.inv_t);
                if (w < p.w_min || place(l, i) < last) w = 0;
            }
            const uint64_t inc = before + scan(w);
            if (w && inc > draw && inc - w <= draw) {
                s_at = i;
                s_wt = w;
            }
            if (tid == kPickThreads - 1) s_before = inc;
            __syncthreads();
            before = s_before;
            if (s_at >= 0) break;
        }
        token = max(s_at, 0);
    }
    if (tid == 0) {
        a.token[b] = token;
        if (a.prob) a.prob[b] = total ? (float)((double)s_wt / (double)total) : 0.0f;
    }
    if (a.x_next) {
        const int d = a.d;
        const size_t r = (size_t)token;
        for (int wd = tid; wd < d / 8; wd += kPickThreads) {
            const uint32_t code = a.embed.q[r * (size_t)(d / 8) + wd];
            const size_t g = r * (size_t)(d / kGroup) + wd / 8;
            *(bf16x8*)(a.x_next + (size_t)b * d + 8 * (size_t)wd) =
                dequant8(code, dq_scale(a.embed.scale[g]), bf16_to_f32(a.embed.bias[g]));
        }
    }
}

}  // namespace

// Logits per chunk: enough chunks for the chip, at most kSampleMaxChunks a row.
int sample_chunk(int V, int B) {
    int chunk = 2048;
    while ((V + chunk - 1) / chunk > kSampleMaxChunks || (int64_t)B * ((V + chunk - 1) / chunk) > 2048) {
        if (chunk >= 16384 && (V + chunk - 1) / chunk <= kSampleMaxChunks) break;
        chunk *= 2;
    }
    return chunk;
}

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
    const dim3 grid(a.n_chunks, a.B);
    hipError_t e;
    sample_max_kernel<<<grid, kThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    trace_point(s);
    sample_hist_kernel<<<grid, kThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    trace_point(s);
    sample_gather_kernel<<<grid, kThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    trace_point(s);
    sample_pick_kernel<<<a.B, kPickThreads, 0, s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
