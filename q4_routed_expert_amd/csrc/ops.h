// ops.h -- launchers of the operators around the MoE layer (scored routing,
// 4-bit products for a few rows, sampling, residual + RMS norm), shared by
// abi.hip and their translation units.
#pragma once
#include "internal.h"

namespace q4moe {

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

// y = W x for a few token rows (moe_linear).
struct LinearArgs {
    Q4 w;                     // [N][K]
    const uint16_t* x;        // bf16 [T][K]
    void* y;                  // fp32 or bf16 [T][N]
    int T, N, K;
    bool out_bf16;
};
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);

}  // namespace q4moe
