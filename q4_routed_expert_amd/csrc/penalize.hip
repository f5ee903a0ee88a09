// penalize.hip -- penalties for repeated tokens, sparse biases and a bit mask on rows of
// logits (moe_penalize), the step between an output head and the sampler.  Per logit l of
// token v, with seen = v is among the row's tokens and n = how often among its answer:
//
//   l <- seen ? (l > 0 ? l / repetition : l * repetition) : l
//   l <- l - frequency n - presence [n > 0] + the row's biases of v
//   l <- allowed(v) ? l : -inf
//
// A work group owns a chunk of the vocabulary of one row: it reads the row's tokens, counts
// those of its chunk in LDS (whole numbers: their order does not matter), then passes once
// over the chunk's logits.  Bound by HBM: 8 bytes per logit; the tokens are read once per
// chunk, from L2.
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kSeen = 0x80000000u;  // the top bit of a counter: seen at all

__global__ __launch_bounds__(kThreads) void penalize_kernel(const PenalizeArgs a) {
    extern __shared__ uint32_t count[];
    const int chunk = 1 << a.chunk_sh, v0 = (int)blockIdx.x << a.chunk_sh, b = blockIdx.y;
    const int V = a.V, n = min(chunk, V - v0), tid = threadIdx.x;
    for (int i = tid; i < n; i += kThreads) count[i] = 0u;
    __syncthreads();
    if (a.tokens) {
        const int total = min(max(a.n_tokens ? a.n_tokens[b] : a.stride, 0), a.stride);
        const int prompt = a.n_prompt ? a.n_prompt[b] : 0;
        const int32_t* tok = a.tokens + (size_t)b * a.stride;
        for (int i = tid; i < total; i += kThreads) {
            const uint32_t at = (uint32_t)tok[i] - (uint32_t)v0;  // (a negative id is far out)
            if (at < (uint32_t)n && tok[i] >= 0) {
                if (i >= prompt) atomicAdd(&count[at], 1u);
                else atomicOr(&count[at], kSeen);
            }
        }
        __syncthreads();
    }
    const float rep0 = a.repetition ? a.repetition[b] : a.repetition_all;
    const float rep = rep0 > 0.0f ? rep0 : 1.0f;  // (NaN too)
    const float freq = a.frequency ? a.frequency[b] : a.frequency_all;
    const float pres = a.presence ? a.presence[b] : a.presence_all;
    const size_t base = (size_t)b * V;
    for (int i = tid; i < n; i += kThreads) {
        const int v = v0 + i;
        float l = a.logits[base + v];
        const uint32_t m = count[i];
        if (m) {
            l = l > 0.0f ? l / rep : l * rep;
            const uint32_t times = m & ~kSeen;
            if (times) l = l - freq * (float)times - pres;
        }
        for (int j = 0; j < a.n_bias; ++j)
            if (a.bias_ids[(size_t)b * a.n_bias + j] == v) l += a.bias[(size_t)b * a.n_bias + j];
        if (a.mask && !((a.mask[(size_t)b * a.mask_words + (v >> 5)] >> (v & 31)) & 1u)) l = -INFINITY;
        a.out[base + v] = l;
    }
}

}  // namespace

hipError_t launch_penalize(const PenalizeArgs& a0, hipStream_t s) {
    PenalizeArgs a = a0;
    a.chunk_sh = 12;
    const int chunk = 1 << a.chunk_sh;
    penalize_kernel<<<dim3((a.V + chunk - 1) / chunk, a.B), kThreads, chunk * sizeof(uint32_t), s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
