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
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);  // (-0.0 + 0.0 = +0.0)
    const uint32_t sign = (uint32_t)((int32_t)(uint32_t)(u >> 32) >> 31);  // all ones: negative
    const uint32_t hi = (uint32_t)(u >> 32) ^ (sign | 0x80000000u), lo = (uint32_t)u ^ sign;
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ double readlane_f64(double v, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ double dpp_f64(double v) {  // 0 where no lane is moved here
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRows, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xF, true);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// Sum over the wave (fixed order), returned to every lane.
__device__ __forceinline__ double wave_sum_f64(double v) {
    v += dpp_f64<0x111>(v);       // row_shr 1, 2, 4, 8: lane 15 of a row has its sum
    v += dpp_f64<0x112>(v);
    v += dpp_f64<0x114>(v);
    v += dpp_f64<0x118>(v);
    v += dpp_f64<0x142, 0xA>(v);  // row_bcast 15
    v += dpp_f64<0x143, 0xC>(v);  // row_bcast 31
    return readlane_f64(v, 63);
}

__device__ __forceinline__ float wave_max_f32(float v) {
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
    auto lane = [&](int i) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i)); };
    return fmaxf(fmaxf(lane(0), lane(16)), fmaxf(lane(32), lane(48)));
}

// exp(-x) for 0 <= x <= 700, else 0 (the header's bound on scores): x = n ln 2 - r with
// |r| <= ln 2 / 2, exp(r) = 1 + r g(r) with g the polynomial of degree 10 through
// (exp(r) - 1) / r at the eleven Chebyshev nodes of the interval (error below 2^-56),
// and 2^-n by the exponent field.
__device__ __forceinline__ double exp_neg(double x) {
    constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: the sum's low bits are the integer
    const double t = fma_const(x, 1.4426950408889634, kMagic);
    const double n = t - kMagic;
    double r = __builtin_fma(n, 0.69314718055994529, -x);  // ln 2 in two parts
    r = __builtin_fma(n, 2.3190468138462996e-17, r);
    double e = 2.5105252864022e-08;
    e = fma_const(e, r, 2.7626348719601085e-07);
    e = fma_const(e, r, 2.7557254891675844e-06);
    e = fma_const(e, r, 2.48015043661086e-05);
    e = fma_const(e, r, 0.00019841269875881047);
    e = fma_const(e, r, 0.0013888888932477204);
    e = fma_const(e, r, 0.008333333333325376);
    e = fma_const(e, r, 0.04166666666657314);
    e = fma_const(e, r, 0.16666666666666674);
    e = fma_const(e, r, 0.5000000000000006);
    e = __builtin_fma(e, r, 1.0);
    e = __builtin_fma(e, r, 1.0);
    const uint64_t u = (uint64_t)__double_as_longlong(e) - ((uint64_t)__double_as_longlong(t) << 52);
    return x <= 700.0 ? __longlong_as_double((long long)u) : 0.0;  // (NaN: 0)
}

// 1 / d for 1 <= d <= 256: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double reciprocal(double d) {
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

// The two largest (a >= b) of two such pairs.
__device__ __forceinline__ void merge_top2(double& a, double& b, double oa, double ob) {
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
}

// The wave's own LDS writes before, its reads after (no other wave's).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Selects one token's experts; lane s < k returns slot s.  s_v: 256 doubles of the wave's.
template <bool SIGMOID>
__device__ __forceinline__ void wave_select(const float* __restrict__ lrow, const ScoreArgs& a,
                                            int lane, double* s_v, int* out_e, float* out_w) {
    const int E = a.E, e0 = 4 * lane;
    float l[4], bal[4];
    double score[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = e0 + i < E ? e0 + i : 0;  // clamped, valid
        l[i] = lrow[e];
        bal[i] = a.balance ? a.balance[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = e0 + i < E ? l[i] : -INFINITY;
    if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double e = exp_neg(fabs((double)l[i])), y = reciprocal(1.0 + e);
            score[i] = l[i] >= 0.0f ? y : l[i] > -INFINITY ? e * y : 0.0;
        }
    } else {
        const float m = wave_max_f32(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (an infinite maximum: 0 apart from itself)
            score[i] = !(l[i] > -INFINITY) ? 0.0 : l[i] == m ? 1.0 : exp_neg((double)m - (double)l[i]);
        const double sum = wave_sum_f64((score[0] + score[1]) + (score[2] + score[3]));
        const double y = sum > 0.0 ? reciprocal(sum) : 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) score[i] *= y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = l[i] > -INFINITY && fabsf(bal[i]) < INFINITY ? score[i] + (double)bal[i] : -INFINITY;
    uint64_t key[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) key[i] = e0 + i < E ? order_key(v[i]) : 0ull;
    if (a.n_groups > 1) {  // uniform
        const int per = E / a.n_groups, sh = __builtin_ctz(per) - 2;
        uint64_t kept = 0;
        auto rank_groups = [&](double mine, int group, int step) {
            int rank = 0;
            for (int g = 0; g < a.n_groups; ++g) {
                const double o = readlane_f64(mine, g << step);
                rank += o > mine || (o == mine && g < group);
            }
            return rank < a.top_groups;
        };
        if (sh >= 0 && per == 4 << sh) {  // a group is 2^sh neighbouring lanes
            double p = fmax(v[0], v[1]), q = fmin(v[0], v[1]);
            merge_top2(p, q, fmax(v[2], v[3]), fmin(v[2], v[3]));
            if (sh > 0) merge_top2(p, q, dpp_f64<0xB1>(p), dpp_f64<0xB1>(q));    // quad_perm 1,0,3,2
            if (sh > 1) merge_top2(p, q, dpp_f64<0x4E>(p), dpp_f64<0x4E>(q));    // quad_perm 2,3,0,1
            if (sh > 2) merge_top2(p, q, dpp_f64<0x141>(p), dpp_f64<0x141>(q));  // row_half_mirror
            if (sh > 3) merge_top2(p, q, dpp_f64<0x140>(p), dpp_f64<0x140>(q));  // row_mirror
            if (sh > 4) merge_top2(p, q, __shfl_xor(p, 16, kWave), __shfl_xor(q, 16, kWave));
            const double mine = a.group_top == 1 || q == -INFINITY ? p : p + q;
            if (!rank_groups(mine, lane >> sh, sh)) key[0] = key[1] = key[2] = key[3] = 0;
        } else {  // any size: lane g reads group g's values from LDS
#pragma unroll
            for (int i = 0; i < 4; ++i) s_v[e0 + i] = v[i];
            wave_lds_fence();
            double p = -INFINITY, q = -INFINITY;
            if (lane < a.n_groups)
                for (int i = 0; i < per; ++i) merge_top2(p, q, s_v[lane * per + i], -INFINITY);
            const double mine = a.group_top == 1 || q == -INFINITY ? p : p + q;
            kept = __ballot(rank_groups(mine, lane, 0) && lane < a.n_groups);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int g = (e0 + i) / per;
                if (g >= a.n_groups || !((kept >> g) & 1ull)) key[i] = 0;
            }
            wave_lds_fence();
        }
    }
    // the scores by expert, 0 where the expert is out
#pragma unroll
    for (int i = 0; i < 4; ++i) s_v[e0 + i] = v[i] > -INFINITY ? score[i] : 0.0;
    wave_lds_fence();
    // each lane's experts in order, equal ones by index (neighbours are exchanged only
    // where the later one is larger); their numbers 0 .. 3 then go into the bytes of `at`
    uint32_t num[4] = {0, 1, 2, 3};
    auto exchange = [&](int i) {
        const bool swap = key[i + 1] > key[i];
        const uint64_t h = swap ? key[i + 1] : key[i];
        key[i + 1] = swap ? key[i] : key[i + 1];
        key[i] = h;
        const uint32_t m = swap ? num[i + 1] : num[i];
        num[i + 1] = swap ? num[i] : num[i + 1];
        num[i] = m;
    };
    exchange(0);
    exchange(1);
    exchange(0);
    exchange(2);
    exchange(1);
    exchange(0);
    uint32_t at = num[0] | num[1] << 8 | num[2] << 16 | num[3] << 24;
    auto umax = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
    int my_e = 0;
#pragma unroll
    for (int s = 0; s < kMaxTopK; ++s) {
        if (s < a.k) {  // uniform
            const uint32_t hi = (uint32_t)(key[0] >> 32), lo = (uint32_t)key[0];
            const uint32_t mh = wave_reduce_u32(hi, umax);
            uint64_t best = __ballot(hi == mh);
            if (best & (best - 1)) {
                const uint32_t ml = wave_reduce_u32(hi == mh ? lo : 0u, umax);
                best = __ballot(hi == mh && lo == ml);
            }
            const int win = (int)__builtin_ctzll(best);  // the lowest expert with the largest key
            const int e = 4 * win + (__builtin_amdgcn_readlane((int)at, win) & 3);
            if (s == lane) my_e = e;
            if (lane == win) {
                key[0] = key[1];
                key[1] = key[2];
                key[2] = key[3];
                key[3] = 0;
                at >>= 8;
            }
        }
    }
    double w = lane < a.k ? s_v[my_e] : 0.0;
    if (a.renorm) {
        const double sum = wave_sum_f64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    *out_e = my_e;
    *out_w = (float)(w * (double)a.scale);
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

// The whole sort for a few tokens by one work group, in one launch: wave w selects for
// token w; a mask of tokens per expert then gives counts (its population) and places (the
// population below a token); the first wave scans counts, 32-row tiles and 128-row tiles
// over the experts.  One token a wave: 1 / 8 / 16 tokens of 256 sigmoid scores in groups
// take 4.8 / 6.2 / 8.1 us against 9.0 / 9.9 / 9.8 of the three launches (graph replays);
// two tokens a wave, at 32, took 15.3 against 11.6.
constexpr int kSmallWaves = 16;
constexpr int kSmallTokens = kSmallWaves;

template <bool SIGMOID>
__global__ __launch_bounds__(64 * kSmallWaves) void route_small_kernel(const ScoreArgs a, const moe_routing r) {
    __shared__ double s_v[kSmallWaves][kMaxExperts];
    __shared__ uint32_t s_mask[kMaxExperts];
    __shared__ int s_off[kMaxExperts], s_b32[kMaxExperts], s_b128[kMaxExperts];
    __shared__ int s_sel[kSmallTokens * kMaxTopK];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int T = a.T, E = a.E, k = a.k;
    if (tid < kMaxExperts) s_mask[tid] = 0;
    __syncthreads();
    if (wave < T) {
        int e;
        float w;
        wave_select<SIGMOID>(a.logits + (size_t)wave * E, a, lane, s_v[wave], &e, &w);
        if (lane < k) {
            a.idx[wave * k + lane] = e;
            a.w[wave * k + lane] = w;
            s_sel[wave * k + lane] = e;
            atomicOr(&s_mask[e], 1u << wave);
        }
    }
    __syncthreads();
    if (wave == 0) {
        int c[4], at[3] = {0, 0, 0}, sum[3] = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = 4 * lane + i < E ? __popc(s_mask[4 * lane + i]) : 0;
            sum[0] += c[i];
            sum[1] += (c[i] + kBlockRows - 1) / kBlockRows;
            sum[2] += (c[i] + kTileRows - 1) / kTileRows;
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            int v = sum[q];
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int x = __shfl_up(v, o, kWave);
                if (lane >= o) v += x;
            }
            at[q] = v - sum[q];
            sum[q] = v;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (4 * lane + i < E) {
                s_off[4 * lane + i] = at[0];
                s_b32[4 * lane + i] = at[1];
                s_b128[4 * lane + i] = at[2];
            }
            at[0] += c[i];
            at[1] += (c[i] + kBlockRows - 1) / kBlockRows;
            at[2] += (c[i] + kTileRows - 1) / kTileRows;
        }
        if (lane == 63) {
            r.offsets[E] = sum[0];
            *r.n_blocks = sum[1];
            *r.n_tiles = sum[2];
        }
    }
    __syncthreads();
    if (tid < E) {
        const int c = __popc(s_mask[tid]), o = s_off[tid];
        r.counts[tid] = c;
        r.offsets[tid] = o;
        for (int j = 0; j * kBlockRows < c; ++j) {
            r.block_map[2 * (s_b32[tid] + j)] = tid;
            r.block_map[2 * (s_b32[tid] + j) + 1] = o + kBlockRows * j;
        }
        for (int j = 0; j * kTileRows < c; ++j) {
            r.tile_map[2 * (s_b128[tid] + j)] = tid;
            r.tile_map[2 * (s_b128[tid] + j) + 1] = o + kTileRows * j;
        }
    }
    if (tid < T * k) {
        const int e = s_sel[tid], pos = s_off[e] + __popc(s_mask[e] & ((1u << (tid / k)) - 1u));
        r.perm[pos] = tid;
        r.inv_perm[tid] = pos;
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

bool route_is_small(int T) { return T <= kSmallTokens; }

hipError_t launch_route_small(const ScoreArgs& a, const moe_routing* r, hipStream_t s) {
    if (a.sigmoid) route_small_kernel<true><<<1, 64 * kSmallWaves, 0, s>>>(a, *r);
    else route_small_kernel<false><<<1, 64 * kSmallWaves, 0, s>>>(a, *r);
    trace_point(s);
    return hipGetLastError();
}

}  // namespace q4moe
