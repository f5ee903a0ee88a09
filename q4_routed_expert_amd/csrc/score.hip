// score.hip -- expert selection of moe_route_scored: softmax or sigmoid scores,
// a balance bias that steers the selection only, expert groups, top-k, and
// renormalised, scaled weights.
//
// A selection decides between scores, so the scores it compares are computed in
// 64 bits: near a border 32 bits would let the rounding of exp decide, and two
// implementations of the same routing would send a token to different experts.
// The vector ALUs run fp64 at the fp32 rate, so this costs registers, not rate.
//
// One wave per token; lane l holds experts 4l .. 4l + 3, so lane order is expert
// order and a ballot finds the lowest expert among equals.  A 64-bit maximum
// over the wave is one 32-bit reduction of the keys' upper words; the lower
// words are reduced only if two lanes share the largest upper word (20 mantissa
// bits: about one round in 10^4).
#include "ops.h"

namespace q4moe {
namespace {

constexpr int kWaves = 4;  // tokens per work group

// Order-preserving 64-bit key: a larger value has a larger key, -0.0 = +0.0.
// Key 0 is below the key of every value, minus infinity included.
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double readlane_f64(double v, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
    return v;
}

// Group scores from the selection values of one token in LDS (lane g: group g):
// the sum of the group's best `group_top` live values, minus infinity if it has
// none.
__device__ __forceinline__ double group_score(const double* s_v, int g, int per, int group_top) {
    double a = -INFINITY, b = -INFINITY;
    for (int i = 0; i < per; ++i) {
        const double v = s_v[g * per + i];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
    }
    return group_top == 1 || b == -INFINITY ? a : a + b;
}

// Selects one token's experts; lane s < k returns slot s.
template <bool SIGMOID>
__device__ __forceinline__ void wave_select(const float* __restrict__ lrow, const ScoreArgs& a,
                                            int lane, double* s_v, int* out_e, float* out_w) {
    const int E = a.E;
    float l[4];
    double score[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = 4 * lane + i < E ? lrow[4 * lane + i] : -INFINITY;
    if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < 4; ++i) score[i] = l[i] > -INFINITY ? 1.0 / (1.0 + exp(-(double)l[i])) : 0.0;
    } else {
        const float m = wave_max_f32(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            score[i] = !(l[i] > -INFINITY) ? 0.0 : l[i] == m ? 1.0 : exp((double)l[i] - (double)m);
            sum += score[i];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float b = a.balance && 4 * lane + i < E ? a.balance[4 * lane + i] : 0.0f;
        v[i] = l[i] > -INFINITY && fabsf(b) < INFINITY ? score[i] + (double)b : -INFINITY;
    }
    uint64_t key[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) key[i] = 4 * lane + i < E ? order_key(v[i]) : 0ull;
    if (a.n_groups > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s_v[4 * lane + i] = v[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // this wave's LDS only
        __builtin_amdgcn_wave_barrier();
        const int per = E / a.n_groups;
        const double mine = lane < a.n_groups ? group_score(s_v, lane, per, a.group_top) : -INFINITY;
        int rank = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const double o = readlane_f64(mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        const uint64_t kept = __ballot(lane < a.n_groups && rank < a.top_groups);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = (4 * lane + i) / per;
            if (g >= a.n_groups || !((kept >> g) & 1ull)) key[i] = 0ull;
        }
    }
    auto umax = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
    int my_e = 0;
    double my_w = 0.0, sum = 0.0;
#pragma unroll
    for (int s = 0; s < kMaxTopK; ++s) {
        if (s < a.k) {  // uniform
            uint64_t h = key[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < 4; ++i)
                if (key[i] > h) {
                    h = key[i];
                    at = i;
                }
            const uint32_t hi = (uint32_t)(h >> 32), lo = (uint32_t)h;
            const uint32_t mh = wave_reduce_u32(hi, umax);
            uint64_t best = __ballot(hi == mh);
            if (best & (best - 1)) {
                const uint32_t ml = wave_reduce_u32(hi == mh ? lo : 0u, umax);
                best = __ballot(hi == mh && lo == ml);
            }
            const int win = (int)__builtin_ctzll(best);  // the lowest expert with the largest key
            const double sc = at == 0 ? score[0] : at == 1 ? score[1] : at == 2 ? score[2] : score[3];
            const double vv = at == 0 ? v[0] : at == 1 ? v[1] : at == 2 ? v[2] : v[3];
            const double w = readlane_f64(vv > -INFINITY ? sc : 0.0, win);
            const int e = 4 * win + __builtin_amdgcn_readlane(at, win);
            if (lane == win) {
#pragma unroll
                for (int i = 0; i < 4; ++i) key[i] = i == at ? 0ull : key[i];
            }
            sum += w;
            if (s == lane) {
                my_e = e;
                my_w = w;
            }
        }
    }
    if (a.renorm) my_w = sum > 0.0 ? my_w / sum : 0.0;
    *out_e = my_e;
    *out_w = (float)(my_w * (double)a.scale);
}

template <bool SIGMOID>
__global__ __launch_bounds__(64 * kWaves) void select_kernel(const ScoreArgs a) {
    __shared__ double s_v[kWaves][kMaxExperts];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * kWaves + wave;
    if (t >= a.T) return;
    int e;
    float w;
    wave_select<SIGMOID>(a.logits + (size_t)t * a.E, a, lane, s_v[wave], &e, &w);
    if (lane < a.k) {
        a.idx[(size_t)t * a.k + lane] = e;
        a.w[(size_t)t * a.k + lane] = w;
        atomicAdd(&a.blk_counts[(size_t)(t / MOE_ROUTE_BLOCK) * a.E + e], 1);
    }
}

}  // namespace

hipError_t launch_select(const ScoreArgs& a, hipStream_t s) {
    const dim3 grid((a.T + kWaves - 1) / kWaves);
    if (a.sigmoid) select_kernel<true><<<grid, 64 * kWaves, 0, s>>>(a);
    else select_kernel<false><<<grid, 64 * kWaves, 0, s>>>(a);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
