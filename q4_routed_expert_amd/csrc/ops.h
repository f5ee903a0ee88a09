// ops.h -- launchers of the operators around the MoE layer (scored routing,
// 4-bit products for a few rows, sampling, residual + RMS norm, 8-bit products,
// rows into expert order and back, penalties on logits), shared by abi.hip and
// their translation units.
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
    float* y8_scale;          // [T][ceil(d/group)], with y8
    int T, d;
    int group;                // 64 or 128
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

// Products in e4m3 (moe_linear_scaled, moe_experts_scaled).
struct ProductArgs {
    const uint8_t* w;         // [E][parts][N][K], parts = 2 when gated
    const float* w_scale;     // [E][parts][ceil(N/128)][ceil(K/128)]
    const uint8_t* x;         // [rows][K]
    const float* x_scale;     // [rows][ceil(K/128)]
    void* y;                  // fp32 or bf16 [rows][N], or e4m3 when gated
    float* y_scale;           // [rows][ceil(N/128)] when gated
    int rows, N, K;           // N: rows of one part
    bool gated, out_bf16;
    bool stream;              // matrices are read once (launch_product sets it)
    // expert-sorted rows (E = 1 and NULL otherwise)
    int E;
    const int32_t* offsets;   // [E + 1]
    const int32_t* map;       // (expert, first row) per tile
    const int32_t* n_map;
    int map_bound;            // host upper bound on *n_map
    const int32_t* map128;    // the same for tiles of 128 rows
    const int32_t* n_map128;
    int map128_bound;
};
hipError_t launch_product(const ProductArgs& a, hipStream_t s);

// Rows into expert order and back (moe_dispatch, moe_combine, moe_combine_grad).
struct SortArgs {
    const int32_t* inv_perm;  // [T][k]
    int pieces;               // threads a token (the launchers set it)
    int T, k, d;
    const uint16_t* x;        // dispatch: bf16 [T][d]
    void* rows_out;           // bf16 or e4m3 [T*k][d] (combine_grad: d_rows)
    float* scale_out;         // dispatch in e4m3: [T*k][ceil(d/128)], or NULL
    const uint16_t* rows;     // combine, combine_grad: bf16 [T*k][d]
    const float* w;           // [T][k] or NULL (all 1)
    const uint16_t* base;     // combine: bf16 [T][d] or NULL
    uint16_t* y;              // combine: bf16 [T][d]
    const uint16_t* dy;       // combine_grad: bf16 [T][d]
    float* d_w;               // combine_grad: [T][k]
};
hipError_t launch_dispatch(const SortArgs& a, hipStream_t s);
hipError_t launch_combine(const SortArgs& a, hipStream_t s);
hipError_t launch_combine_grad(const SortArgs& a, hipStream_t s);

// Penalties, biases and a mask on logits (moe_penalize).
struct PenalizeArgs {
    const float* logits;      // [B][V]
    float* out;               // [B][V], may be logits
    int B, V;
    const int32_t* tokens;    // [B][stride] or NULL
    const int32_t* n_tokens;  // [B] or NULL (all stride)
    const int32_t* n_prompt;  // [B] or NULL (0)
    int stride;
    const float* repetition;  // [B] or NULL (then repetition_all), and so on
    const float* frequency;
    const float* presence;
    float repetition_all, frequency_all, presence_all;
    const int32_t* bias_ids;  // [B][n_bias]
    const float* bias;        // [B][n_bias]
    int n_bias;
    const uint32_t* mask;     // [B][mask_words] or NULL
    int mask_words;
};
hipError_t launch_penalize(const PenalizeArgs& a, hipStream_t s);

}  // namespace q4moe
