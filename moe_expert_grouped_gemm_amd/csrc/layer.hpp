// layer.hpp -- internal launcher interface of the operators around the expert
// GEMM: residual RMS norm, router, whole layer for a few tokens.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ptgg {

// ------------------------------------------------------------------ RMS norm
enum NormCodes { kCodesNone = 0, kCodesMx = 1, kCodesRows = 2 };

struct NormFwdParams {
    const uint16_t *x;        // [rows, cols] bf16
    const void *residual;     // [rows, cols] stream type, or null
    const uint16_t *weight;   // [cols] bf16
    void *residual_out;       // [rows, cols] stream type, or null
    uint16_t *y;              // [rows, cols] bf16, or null
    uint8_t *q;               // [rows, cols] E4M3 codes, or null
    void *scales;             // E8M0 [rows, cols/32] or fp32 [rows]
    float *rstd;              // [rows], or null
    int64_t rows;
    int cols;
    float eps;
    int f32;                  // the residual stream is fp32 (else bf16)
    int codes;                // NormCodes
};
hipError_t launch_rmsnorm_fwd(const NormFwdParams &p, hipStream_t s);

struct NormBwdParams {
    const uint16_t *dy;       // [rows, cols] bf16
    const void *s;            // [rows, cols] stream type: the forward's residual_out
    const uint16_t *weight;
    const float *rstd;
    const void *dres;         // [rows, cols] stream type, or null
    void *ds;                 // [rows, cols] stream type
    float *dweight;           // [cols], or null
    float *partials;          // workspace: norm_bwd_parts(rows) x [cols], or null for one part
    int64_t rows;
    int cols;
    int f32;
    int accumulate;
};
// Row parts whose weight gradients are summed apart (1: none needed).
int norm_bwd_parts(int64_t rows);
hipError_t launch_rmsnorm_bwd(const NormBwdParams &p, hipStream_t s);
// Longest row the norm kernels hold in registers.
constexpr int kNormMaxCols = 32768;

// ------------------------------------------------------------------ router
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 16;
constexpr int kRouteChunk = 64;           // tokens whose order one workgroup finds at a time
constexpr int kRouteMaxParts = 256;
constexpr uint32_t kErrNanLogit = 16u;    // sticky device error bit

struct RouteParams {
    const void *logits;       // [T, E] fp32 or bf16
    const float *bias;        // [E] added to the sigmoid scores for the choice, or null
    int32_t *topk_ids;        // [T, k]
    float *topk_weights;      // [T, k]
    int64_t *lens;            // [E]
    int32_t *row_of;          // [T, k]
    int32_t *token_of;        // [T * k]
    uint16_t *counts;         // workspace: [parts][route_pitch(E)] tokens of each part that chose an expert
    uint32_t *err;
    int64_t T;
    int E, k;
    int bf16;                 // logits are bf16
    int sigmoid;
    int renorm;
    float scale;
};
// The few-token layer's list of the expert matrices to stream: plan[0] blocks
// of at most `cap` <= 16 rows of one expert, from plan + 4.  An expert's `of`
// blocks follow each other from the list's place `first`.
struct FewBlock {
    int expert, row0, rows;
    uint16_t first, of;
    uint8_t token[16];
};
struct RoutePlan {
    int *plan;
    int cap;
};
int route_parts(int64_t T);
// Experts in a row of the counts, which are read 8 at a time.
__host__ __device__ constexpr int route_pitch(int E) { return (E + 7) & ~7; }
hipError_t launch_moe_route(const RouteParams &p, hipStream_t s);
// At most kRouteChunk tokens; also writes the plan.
hipError_t launch_moe_route_plan(const RouteParams &p, const RoutePlan &plan, hipStream_t s);

struct RouteBwdParams {
    const void *logits;
    const int32_t *topk_ids;
    const float *dweights;    // [T, k]
    void *dlogits;            // [T, E], the logits' type
    int64_t T;
    int E, k;
    int bf16, sigmoid, renorm;
    float scale;
};
hipError_t launch_moe_route_bwd(const RouteBwdParams &p, hipStream_t s);

// ------------------------------------------------------------------ the layer for a few tokens
enum FewWeights { kFewBf16 = 0, kFewMxfp8 = 1, kFewMxfp4 = 2 };
constexpr int kFewMaxTokens = kRouteChunk;
constexpr int64_t kFewMaxWidth = 16384;   // hidden and inner sizes

struct FewParams {
    const uint16_t *x;        // [T, H] bf16
    const uint8_t *w1, *w1s;  // [E, 2I, H] (gate | up) and its E8M0 scales
    const uint8_t *w2, *w2s;  // [E, H, I]
    uint16_t *out;            // [T, H] bf16
    RouteParams route;        // its lens, row_of and token_of lie in the workspace
    int *plan;                // workspace: 4 ints and T k blocks at most
    uint16_t *h;              // workspace [T k, I] bf16
    float *y;                 // workspace [T k, H]
    int T, E, H, I, k;
    int weights;              // FewWeights
    float swiglu_limit;
};
hipError_t launch_few_tokens(const FewParams &p, hipStream_t s);

}  // namespace ptgg
