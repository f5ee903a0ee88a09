// ops.h -- launchers of the operators around the MoE layer (scored routing,
// 4-bit products for a few rows, sampling, residual + RMS norm), shared by
// abi.hip and their translation units.
#pragma once
#include "internal.h"

namespace q4moe {

// a * b + c with c in scalar registers (the compiler keeps such constants in vector
// registers and copies them for its two-operand form, one more instruction a step).
__device__ __forceinline__ double fma_const(double a, double b, double c) {
    double d;
    #if defined(__HIP_DEVICE_COMPILE__)
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
#else
    d = __builtin_fma(a, b, c);
#endif
    return d;
}


// y = norm(x + residual) (moe_add_norm).
struct NormArgs {
    const uint16_t* x;        // bf16 [T][d]
    const void* residual;     // bf16 or fp32 [T][d], or NULL
    void* residual_out;       // the same type, or NULL; may be residual
    const uint16_t* weight;   // bf16 [d]
    uint16_t* y;              // bf16 [T][d], or NULL
    uint8_t* y8;              // e4m3 [T][d], or NULL
    float* y8_scale;          // [T][d/64], with y8
    int T, d;
    float eps, w_add;         // the weight used is weight + w_add
    bool res_f32;
};
hipError_t launch_add_norm(const NormArgs& a, hipStream_t s);

// Expert selection of moe_route_scored (the top-k step of routing).
struct ScoreArgs {
    const float* logits;      // [T][E]
    const float* balance;     // [E] or NULL
    int T, E, k;
    int n_groups, top_groups, group_top;
    bool sigmoid, renorm;
    float scale;
    int32_t* idx;             // [T][k]
    float* w;                 // [T][k]
    int32_t* blk_counts;      // [ceil(T/MOE_ROUTE_BLOCK)][E], cleared; counts are added
};
hipError_t launch_select(const ScoreArgs& a, hipStream_t s);
// Selection and sort of a few tokens in one launch (blk_counts is not used).
bool route_is_small(int T);
hipError_t launch_route_small(const ScoreArgs& a, const moe_routing* r, hipStream_t s);

// y = W x for a few token rows (moe_linear).
struct LinearArgs {
    Q4 w;                     // [N][K]
    const uint16_t* x;        // bf16 [T][K]
    void* y;                  // fp32 or bf16 [T][N]
    int T, N, K;
    bool out_bf16;
};
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);

// One token per row of logits (moe_sample).
constexpr int kSampleBins = 2048;       // histogram bins of a row
constexpr int kSampleList = 4096;       // tokens a row's list holds
constexpr int kSampleMaxChunks = 512;   // chunks of a row
constexpr int kSampleRowMax = 8192;     // rows up to here take the one-kernel form
struct SampleState {     // what a row's histogram says about its cut
    uint64_t total;      // sum of the histogram (its mass, or with top-k its count)
    uint64_t before;     // mass before the listed bins
    int32_t lo, hi;      // the listed bins
    int32_t reached;     // the target lies in bin hi
    int32_t pad;
};
struct SampleRow {       // one row's parameters
    double inv_t;        // 1 / temperature
    double p;            // top-p
    uint64_t w_min;      // min-p: the smallest kept weight, >= 1
    uint32_t k;          // tokens top-k keeps, 1 .. V
    float u;
    int32_t cut_k, cut_p;  // top-k / top-p are on
};
struct SampleArgs {
    const float* logits;      // [B][V]
    int B, V, d, chunk_sh, n_chunks;
    const float* temperature; // [B] or NULL (then temperature_all), and so on
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    float temperature_all;
    int32_t top_k_all;
    float top_p_all, min_p_all;
    const float* u;           // [B]
    int32_t* token;           // [B]
    float* prob;              // [B] or NULL
    uint16_t* x_next;         // bf16 [B][d] or NULL
    Q4 embed;                 // [V][d]
    // workspace (unused by short rows)
    float* part_max;          // [B][n_chunks]
    uint64_t* chunk_w;        // [B][n_chunks]
    uint64_t* hist;           // [B][kSampleBins]
    uint64_t* list;           // [B][kSampleList]
    uint32_t* list_n;         // [B]
    SampleState* state;       // [B]
    SampleRow* row;           // [B]
};
int sample_chunk_sh(int V, int B);  // log2 of the logits per chunk
hipError_t launch_sample(const SampleArgs& a, hipStream_t s);

}  // namespace q4moe
