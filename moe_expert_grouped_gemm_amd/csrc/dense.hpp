// dense.hpp -- internal launcher interface of the dense operators of an MoE
// block: the matrix product with bias, activation and residual in its epilogue
// and its gradients, the norms around a block with its gate, the experts'
// weighted sum.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ptgg {

// ------------------------------------------------------------------ matrix product
enum LinearOp { kLinFwd = 0, kLinDgrad = 1, kLinWgrad = 2 };
// as pt_act
enum Act { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu2 = 4, kActSwiglu = 5 };
// What becomes of 8 neighbouring sums of the product (finish8 in linear.hip).
enum Finish {
    kFinFwd = 0,      // + bias, saved, activation, + residual
    kFinFwdGlu = 1,   // the same from 8 gates and the 8 ups N/2 columns on
    kFinGrad = 2,     // times the activation's derivative at the saved sums, + residual
    kFinGradGlu = 3,  // the gradients of 8 gates and 8 ups
    kFinPartial = 4   // as they are: fp32 sums of one part of the reduction
};

struct FinishParams {
    const uint16_t *bias;     // [N] bf16, or null
    const void *residual;     // [M, ldo] of out's type, or null
    void *out;                // [M, ldo] bf16 or fp32
    uint16_t *save;           // kFinFwd*: the sums with bias, [M, N] bf16, or null
    const uint16_t *c;        // kFinGrad*: the saved sums, [M, ldo] bf16, or null
    int64_t N;                // columns of the product
    int64_t ldo;              // columns of out
    int finish;
    int act;
    int f32;                  // out and residual are fp32 (else bf16)
    float limit;              // SwiGLU clamp, +inf for none
};

// How the widest tile's work is spread over the CUs (wide_cut in linear_plan.hpp): the
// first `whole` tiles in one piece; each of the `rest` others in `parts` of `main`
// reduction values and a tail, which the first `tails` of them take in one piece,
// the others in `cuts` of `cut` values.  rest = 0: every tile in one piece.
struct WideCut {
    int whole, rest, parts, tails, cuts;
    int64_t main, cut;
    __host__ __device__ int pieces() const { return parts * rest + tails + (rest - tails) * cuts; }
};

// dbias[n] (+)= sum over rows of dy[r, n].  parts > 1: sums of each part's rows in
// partials, [parts][N], joined afterwards.
struct ColsumParams {
    const uint16_t *dy;       // [M, N] bf16
    float *dbias;             // or null: not wanted
    float *partials;
    int64_t M, N;
    int parts;
    int accumulate;
};
int colsum_parts(int64_t M, int64_t N);

// C[m, n] = sum over q < K of A(m, q) B(n, q): forward A = x, B = w; dgrad
// A = dy, B = w by columns; wgrad A = dy and B = x by columns.
struct LinearParams {
    const uint16_t *a, *b;
    int64_t M, N, K;          // of the product as computed
    int64_t lda, ldb;         // elements between rows in memory
    int splits;               // parts of the reduction
    int64_t part;             // reduction values a part (a multiple of 64)
    float *partials;          // workspace: splits x [M, N] fp32, where splits > 1; or the cut's pieces, a tile each
    WideCut cut;              // of the widest tile
    ColsumParams sums;        // wgrad: the bias's gradient
    int join_blocks;          // workgroups of the join that add the product's parts; the others join the column sums
    FinishParams f;
};

// How a product runs: which tile, and in how many parts.
struct LinearPlan {
    int tile;
    int splits;
    int64_t part;
    WideCut cut;
    int64_t partial_bytes;
};
LinearPlan linear_plan(int op, int64_t M, int64_t N, int64_t K);
hipError_t launch_linear(const LinearParams &p, int op, const LinearPlan &plan, hipStream_t s);

// dc = dout * act'(c) over [M, N] (SwiGLU: dout [M, N/2]).
hipError_t launch_act_bwd(const uint16_t *dout, const uint16_t *c, uint16_t *dc, int64_t M, int64_t N, int act,
                          float limit, hipStream_t s);

// ------------------------------------------------------------------ norms around a block
enum BlockGate { kGateNone = 0, kGateCols = 1, kGateRows = 2, kGateFull = 3 };
constexpr int kBlockMaxCols = 16384;      // longest row that the backward holds in registers

struct BlockNormFwdParams {
    const uint16_t *x;        // [rows, cols] bf16: the block's output
    const void *residual;     // [rows, cols] stream type
    const uint16_t *post;     // [cols] bf16, or null (no norm after the block)
    const void *gate;         // bf16 [cols], fp32 [rows] or bf16 [rows, cols], or null
    const uint16_t *pre;      // [cols] bf16, or null (no norm before the next block)
    void *residual_out;       // [rows, cols] stream type
    uint16_t *y;              // [rows, cols] bf16, or null
    uint8_t *q;
    void *scales;
    float *rstd_post, *rstd_pre;   // [rows], or null
    int64_t rows;
    int cols;
    float eps, branch_scale, residual_scale;
    int gate_kind;
    int f32;
    int codes;                // NormCodes
};
hipError_t launch_block_norm_fwd(const BlockNormFwdParams &p, hipStream_t s);

struct BlockNormBwdParams {
    const uint16_t *dy;       // [rows, cols] bf16, or null (no norm before the next block)
    const void *dres;         // [rows, cols] stream type, or null
    const uint16_t *x;
    const void *s;            // the forward's residual_out
    const uint16_t *post;
    const void *gate;
    const uint16_t *pre;
    const float *rstd_post, *rstd_pre;
    uint16_t *dx;             // [rows, cols] bf16
    void *dresidual;          // [rows, cols] stream type
    void *dgate;              // fp32 [cols], fp32 [rows] or bf16 [rows, cols], or null
    float *dpost, *dpre;      // [cols], or null
    float *partials;          // workspace: parts x 2 x [cols]
    int64_t rows;
    int cols;
    float branch_scale, residual_scale;
    int gate_kind;
    int f32;
    int accumulate;
    int sums;                 // dpre, dpost or a gate per column's gradient is wanted
};
int block_norm_parts(int64_t rows, int64_t cols);
hipError_t launch_block_norm_bwd(const BlockNormBwdParams &p, hipStream_t s);

// ------------------------------------------------------------------ experts' weighted sum
struct CombineParams {
    const uint16_t *rows;     // [M, H] bf16
    const float *weights;     // [T, k], or null (ones)
    const int32_t *row_of;    // [T, k]; a value outside [0, M) is no row
    const uint16_t *base;     // [T, H] bf16, or null
    uint16_t *out;            // [T, H] bf16
    int64_t T, M;
    int H, k;
};
hipError_t launch_combine(const CombineParams &p, hipStream_t s);

struct CombineBwdParams {
    const uint16_t *dout;     // [T, H] bf16
    const uint16_t *rows;     // [M, H] bf16, or null where dweights is
    const float *weights;
    const int32_t *row_of;
    uint16_t *drows;          // [M, H] bf16, or null
    float *dweights;          // [T, k], or null
    int64_t T, M;
    int H, k;
};
hipError_t launch_combine_bwd(const CombineBwdParams &p, hipStream_t s);
constexpr int kCombineMaxCols = 32768;

}  // namespace ptgg
