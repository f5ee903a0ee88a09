// penalize.hip -- penalties for repeated tokens, sparse biases and a bit mask on rows of
// logits (moe_penalize), the step between an output head and the sampler.  Per logit l of
// token v, with seen = v is among the row's tokens and n = how often among its answer:
//
//   l <- seen ? (l > 0 ? l / repetition : l * repetition) : l
//   l <- l - frequency n - presence [n > 0] + the row's biases of v
//   l <- allowed(v) ? l : -inf
//
// A work group owns a chunk of the vocabulary of one row: it reads the row's tokens, counts
// those of its chunk in LDS (whole numbers: their order does not matter), then passes once over
// the chunk's logits, and last adds the biases of its tokens, a thread for each (looking for a
// token's biases in the pass instead cost a walk over the list per biased token: 95 us for 64
// rows of 248320 with 100 biases).  Where a token of the chunk has two biases, the chunk's are
// gathered in list order first and compared there.
// Bound by HBM: 8 bytes per logit; the tokens are read once per chunk, from L2.  In place,
// logits that nothing touches are neither read nor written.
// Measured: 64 rows of 248320 with 4000 tokens at most, masks and 100 biases 32 us into a new buffer
// and 28 into that of the call before (a copy of the logits takes 25), in place 25.5; with 32000
// tokens 44, 39 and 34, with 1000 biases 37, 33 and 31; one row 3.8.
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kSeen = 0x80000000u;    // top bits of a counter: seen at all,
constexpr uint32_t kBiased = 0x40000000u;  // has a bias
constexpr uint32_t kTimes = 0x3FFFFFFFu;

// Sixteen bytes at a 4-byte address (rows of odd lengths).
template <typename T>
struct __attribute__((packed, aligned(4))) Four {
    T v[4];
};

// Four logits at `at` of a row; the last ones may lie behind its end.
__device__ __forceinline__ Four<float> load4(const float* row, int at, int n) {
    if (at + 4 <= n) return *(const Four<float>*)(row + at);
    Four<float> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = at + i < n ? row[at + i] : 0.0f;
    return f;
}

// NV pieces of four logits per thread: a chunk is 1024 NV logits.
template <int NV, bool IN_PLACE>
__global__ __launch_bounds__(kThreads) void penalize_kernel(const PenalizeArgs a) {
    constexpr int kChunk = NV * 4 * kThreads;
    __shared__ u32x4 count4[kChunk / 4];
    uint32_t* count = (uint32_t*)count4;
    const int v0 = (int)blockIdx.x * kChunk, b = blockIdx.y, tid = threadIdx.x;
    const int V = a.V, n = min(kChunk, V - v0);
    const float* in = a.logits + (size_t)b * V + v0;
    float* out = a.out + (size_t)b * V + v0;
    const uint32_t* mask = a.mask ? a.mask + (size_t)b * a.mask_words : nullptr;
    __shared__ int twice;  // a token of the chunk has two biases
    Four<float> l[NV];
    uint32_t allowed[NV];
    // in flight while the tokens are counted
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int at = 4 * (tid + kThreads * j);
        if constexpr (!IN_PLACE) l[j] = load4(in, at, n);
        allowed[j] = mask && at < n ? mask[(v0 + at) >> 5] : 0xFFFFFFFFu;
    }
    if (a.tokens || a.n_bias) {
#pragma unroll
        for (int j = 0; j < NV; ++j) count4[tid + kThreads * j] = u32x4{0u, 0u, 0u, 0u};
        if (tid == 0) twice = 0;
        __syncthreads();
    }
    if (a.tokens) {
        const int total = a.n_tokens ? min(max(a.n_tokens[b], 0), a.stride) : a.stride;
        const int prompt = a.n_prompt ? a.n_prompt[b] : 0;
        const int32_t* tok = a.tokens + (size_t)b * a.stride;
        auto add = [&](int32_t id, int i) {
            const uint32_t at = (uint32_t)id - (uint32_t)v0;
            if (id >= 0 && at < (uint32_t)n) {
                if (i >= prompt) atomicAdd(&count[at], 1u);
                else atomicOr(&count[at], kSeen);
            }
        };
        int i = 4 * tid;
        // four loads at a time, as a long history would wait for them one by one
        for (; i + 12 * kThreads + 4 <= total; i += 16 * kThreads) {
            Four<int32_t> t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = *(const Four<int32_t>*)(tok + i + 4 * kThreads * k);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) add(t[k].v[j], i + 4 * kThreads * k + j);
        }
        for (; i + 4 <= total; i += 4 * kThreads) {
            const Four<int32_t> t = *(const Four<int32_t>*)(tok + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) add(t.v[j], i + j);
        }
        for (; i < total; ++i) add(tok[i], i);  // one thread's: the last ones
    }
    const int32_t* ids = a.bias_ids + (size_t)b * a.n_bias;
    for (int i = tid; i < a.n_bias; i += kThreads) {
        const int32_t id = ids[i];
        const uint32_t at = (uint32_t)id - (uint32_t)v0;
        if (id >= 0 && at < (uint32_t)n && (atomicOr(&count[at], kBiased) & kBiased)) twice = 1;
    }
    if (a.tokens || a.n_bias) __syncthreads();
    const float rep0 = a.repetition ? a.repetition[b] : a.repetition_all;
    const float rep = rep0 > 0.0f ? rep0 : 1.0f;  // (NaN too)
    const float freq = a.frequency ? a.frequency[b] : a.frequency_all;
    const float pres = a.presence ? a.presence[b] : a.presence_all;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int at = 4 * (tid + kThreads * j);
        if (at >= n) continue;
        // (v0 + at is a multiple of 4: the four bits are in one word)
        const uint32_t bits = (allowed[j] >> ((v0 + at) & 31)) & 15u;
        u32x4 m = {0u, 0u, 0u, 0u};
        if (a.tokens) m = count4[tid + kThreads * j];
        if constexpr (IN_PLACE) {
            if (bits == 15u && ((m[0] | m[1] | m[2] | m[3]) & ~kBiased) == 0u) continue;
            l[j] = load4(in, at, n);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = l[j].v[i];
            if (m[i] & ~kBiased) {
                const uint32_t times = m[i] & kTimes;
                x = x > 0.0f ? x / rep : x * rep;
                // (one rounding an operation)
                if (times) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, (float)times)), pres);
            }
            l[j].v[i] = (bits >> i) & 1u ? x : -INFINITY;
        }
        if (at + 4 <= n) {
            *(Four<float>*)(out + at) = l[j];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at + i < n) out[at + i] = l[j].v[i];
        }
    }
    if (!a.n_bias) return;
    __syncthreads();  // the work group's logits are stored
    const float* bias = a.bias + (size_t)b * a.n_bias;
    auto allows = [&](uint32_t at) { return !mask || ((mask[(v0 + at) >> 5] >> ((v0 + at) & 31)) & 1u); };
    if (!twice) {
        for (int i = tid; i < a.n_bias; i += kThreads) {
            const uint32_t at = (uint32_t)ids[i] - (uint32_t)v0;
            if (ids[i] >= 0 && at < (uint32_t)n && allows(at)) out[at] += bias[i];
        }
        return;
    }
    // The chunk's biases, in list order, in the place of the counters: (token, place in the list);
    // then the first one of a token adds all of them, in order.
    static_assert(kChunk >= MOE_MAX_BIASES && kChunk <= (1 << 22) && MOE_MAX_BIASES <= 1024, "room for the list");
    __shared__ int found[kThreads / 64];
    int m = 0;
    for (int i0 = 0; i0 < a.n_bias; i0 += kThreads) {
        const int i = i0 + tid, id = i < a.n_bias ? ids[i] : -1;
        const uint32_t at = (uint32_t)id - (uint32_t)v0;
        const bool here = id >= 0 && at < (uint32_t)n;
        const uint64_t lanes = __ballot(here);
        if ((tid & 63) == 0) found[tid >> 6] = (int)__builtin_popcountll(lanes);
        __syncthreads();
        int before = m;
        for (int w = 0; w < kThreads / 64; ++w) {
            if (w < (tid >> 6)) before += found[w];
            m += found[w];
        }
        before += (int)__builtin_popcountll(lanes & ((1ull << (tid & 63)) - 1));
        if (here) count[before] = at << 10 | (uint32_t)i;
        __syncthreads();
    }
    if (tid < ((4 - (m & 3)) & 3)) count[m + tid] = ~0u;  // (no token's)
    __syncthreads();
    for (int q = tid; q < m; q += kThreads) {
        const uint32_t at = count[q] >> 10;
        if (!allows(at)) continue;
        float x = out[at];
        bool first = true;
        for (int k = 0; k < m; k += 4) {
            const u32x4 e = count4[k >> 2];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e[j] >> 10 == at) {
                    if (k + j < q) first = false;
                    else x += bias[e[j] & 1023u];
                }
        }
        if (first) out[at] = x;
    }
}

// The logits stay in the caches for whoever reads them next.  Loads and stores that pass them by make
// this call alone shorter (64 rows of 248320 26.5 us instead of 31.7) and the step longer: with the
// sampler after it 98.7 instead of 96.8, with an argmax 122 instead of 100.
template <int NV>
void launch(const PenalizeArgs& a, hipStream_t s) {
    const dim3 grid((a.V + NV * 4 * kThreads - 1) / (NV * 4 * kThreads), a.B);
    if (a.out == a.logits) penalize_kernel<NV, true><<<grid, kThreads, 0, s>>>(a);
    else penalize_kernel<NV, false><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

// Chunks of 1024, 2048, 4096 and 8192 logits (us, 248320 logits a row, new buffers): larger ones read
// the history less often, smaller ones are more work groups.  4000 tokens: 1 row (2000) 3.9, 4.4, 5.4,
// 7.6; 4 rows 5.7, 6.2, 7.2, 9.4; 16 rows 12.9, 11.6, 12.0, 13.1; 32 rows 20.1, 17.6, 16.8, 17.5; 64
// rows 46, 34, 33, 35.  64 rows with 32000 tokens 83, 57, 44.6, 45.4, 65000 130, 85, 64.4, 62.7,
// 131072 211, 133, 95, 90.
hipError_t launch_penalize(const PenalizeArgs& a, hipStream_t s) {
    const long long logits = (long long)a.B * a.V;
    if (logits >= 8192LL * 1024 && a.tokens && a.stride > 32768) launch<8>(a, s);
    else if (logits >= 4096LL * 1024) launch<4>(a, s);
    else if (logits >= 2048LL * 512) launch<2>(a, s);
    else launch<1>(a, s);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
