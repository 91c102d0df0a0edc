// dense_api.cpp -- the C ABI (include/ptgg.h) of the dense operators of an MoE
// block: matrix product with its epilogue and gradients, norms around a block,
// the experts' weighted sum.  Argument checks and dispatch; nothing here reads
// device memory, allocates or synchronises.
#include "checks.hpp"
#include "dense.hpp"
#include "layer.hpp"

using namespace ptgg;

namespace {

constexpr int64_t kMaxWidth = (int64_t)1 << 17;          // columns and reduction of a product
constexpr int64_t kMaxProduct = (int64_t)1 << 38;        // elements of a matrix
constexpr int64_t kMaxTokens = (int64_t)1 << 36;         // elements of a matrix of rows: a launch stays below 2^32 threads

bool is_act(int act) { return act >= PT_ACT_NONE && act <= PT_ACT_SWIGLU; }

int check_product(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 1 || K < 1) return PT_ERR_INVALID_ARG;
    if (N % 8 || K % 8 || M > kMaxRows || N > kMaxWidth || K > kMaxWidth) return PT_ERR_UNSUPPORTED;
    if (M * N > kMaxProduct || M * K > kMaxProduct) return PT_ERR_UNSUPPORTED;
    return PT_OK;
}

float glu_limit(float v)
{
    const float inf = __builtin_huge_valf();
    return v > 0.0f && v < inf ? v : inf;
}

// The product that an operator computes: rows, columns and reduction.
LinearPlan plan_of(int op, int64_t M, int64_t N, int64_t K)
{
    if (op == PT_OP_FWD) return linear_plan(kLinFwd, M, N, K);
    if (op == PT_OP_DGRAD) return linear_plan(kLinDgrad, M, K, N);
    return linear_plan(kLinWgrad, N, K, M);
}

int64_t colsum_bytes(int64_t M, int64_t N)
{
    const int parts = colsum_parts(M, N);
    return parts > 1 ? (int64_t)parts * N * 4 : 0;
}

int check_block_norm(int64_t rows, int64_t cols, float branch_scale, float residual_scale, int gate_kind, int stream_dtype)
{
    if (rows < 0 || cols < 1 || branch_scale != branch_scale || residual_scale != residual_scale) return PT_ERR_INVALID_ARG;
    if (gate_kind < PT_BLOCK_GATE_NONE || gate_kind > PT_BLOCK_GATE_FULL) return PT_ERR_INVALID_ARG;
    if (stream_dtype != PT_BF16 && stream_dtype != PT_FP32) return PT_ERR_UNSUPPORTED;
    if (cols % 8 || cols > kBlockMaxCols || rows > kMaxRows || rows * cols > kMaxTokens) return PT_ERR_UNSUPPORTED;
    return PT_OK;
}

int check_combine(int64_t T, int64_t M, int64_t H, int64_t k)
{
    if (T < 0 || M < 0 || H < 1 || k < 1) return PT_ERR_INVALID_ARG;
    if (H % 8 || H > kCombineMaxCols || k > PT_MAX_TOPK || T > kMaxRows || M > INT32_MAX || T * H > kMaxTokens)
        return PT_ERR_UNSUPPORTED;
    return PT_OK;
}

}  // namespace

extern "C" {

size_t pt_linear_workspace_size(int op, int64_t M, int64_t N, int64_t K)
{
    if ((op != PT_OP_FWD && op != PT_OP_DGRAD && op != PT_OP_WGRAD) || check_product(M, N, K) != PT_OK) return 0;
    if (M == 0) return 0;
    const LinearPlan plan = plan_of(op, M, N, K);
    return (size_t)(plan.partial_bytes + (op == PT_OP_WGRAD ? colsum_bytes(M, N) : 0));
}

int pt_linear_fwd(const void *x, const void *w, const void *bias, const void *residual, void *out, void *c, int64_t M,
                  int64_t N, int64_t K, int act, int out_dtype, float swiglu_limit, void *workspace,
                  size_t workspace_bytes, void *stream)
{
    const int st = check_product(M, N, K);
    if (st == PT_ERR_INVALID_ARG || !is_act(act) || swiglu_limit != swiglu_limit) return PT_ERR_INVALID_ARG;
    if (st) return st;
    if (out_dtype != PT_BF16 && out_dtype != PT_FP32) return PT_ERR_UNSUPPORTED;
    if (act == PT_ACT_SWIGLU && N % 16) return PT_ERR_UNSUPPORTED;
    if (M == 0) return PT_OK;
    if (!x || !w || !out) return PT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(out, 16) ||
        !aligned(c, 16))
        return PT_ERR_MISALIGNED;
    const LinearPlan plan = plan_of(PT_OP_FWD, M, N, K);
    if (plan.partial_bytes && (!workspace || workspace_bytes < (size_t)plan.partial_bytes)) return PT_ERR_WORKSPACE;
    if (plan.partial_bytes && !aligned(workspace, 16)) return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    LinearParams p = {};
    p.a = (const uint16_t *)x;
    p.b = (const uint16_t *)w;
    p.M = M;
    p.N = N;
    p.K = K;
    p.lda = p.ldb = K;
    p.partials = (float *)workspace;
    p.f.bias = (const uint16_t *)bias;
    p.f.residual = residual;
    p.f.out = out;
    p.f.save = (uint16_t *)c;
    p.f.N = N;
    p.f.ldo = act == PT_ACT_SWIGLU ? N / 2 : N;
    p.f.finish = act == PT_ACT_SWIGLU ? kFinFwdGlu : kFinFwd;
    p.f.act = act;
    p.f.f32 = out_dtype == PT_FP32;
    p.f.limit = glu_limit(swiglu_limit);
    return hip_status(launch_linear(p, kLinFwd, plan, (hipStream_t)stream));
}

int pt_linear_dgrad(const void *dy, const void *w, const void *c, const void *add, void *dx, int64_t M, int64_t N,
                    int64_t K, int act, float swiglu_limit, void *workspace, size_t workspace_bytes, void *stream)
{
    const int st = check_product(M, N, K);
    if (st == PT_ERR_INVALID_ARG || !is_act(act) || swiglu_limit != swiglu_limit) return PT_ERR_INVALID_ARG;
    if (st) return st;
    if (M == 0) return PT_OK;
    if (!dy || !w || !dx || (c != nullptr) != (act != PT_ACT_NONE) || (add && act == PT_ACT_SWIGLU))
        return PT_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(c, 16) || !aligned(add, 16) || !aligned(dx, 16))
        return PT_ERR_MISALIGNED;
    const LinearPlan plan = plan_of(PT_OP_DGRAD, M, N, K);
    if (plan.partial_bytes && (!workspace || workspace_bytes < (size_t)plan.partial_bytes)) return PT_ERR_WORKSPACE;
    if (plan.partial_bytes && !aligned(workspace, 16)) return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    LinearParams p = {};
    p.a = (const uint16_t *)dy;
    p.b = (const uint16_t *)w;
    p.M = M;
    p.N = K;
    p.K = N;
    p.lda = N;
    p.ldb = K;
    p.partials = (float *)workspace;
    p.f.residual = add;
    p.f.out = dx;
    p.f.c = (const uint16_t *)c;
    p.f.N = K;
    p.f.ldo = act == PT_ACT_SWIGLU ? 2 * K : K;
    p.f.finish = act == PT_ACT_SWIGLU ? kFinGradGlu : kFinGrad;
    p.f.act = act;
    p.f.limit = glu_limit(swiglu_limit);
    return hip_status(launch_linear(p, kLinDgrad, plan, (hipStream_t)stream));
}

int pt_linear_wgrad(const void *x, const void *dy, float *main_grad, float *dbias, int64_t M, int64_t N, int64_t K,
                    int accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    const int st = check_product(M, N, K);
    if (st == PT_ERR_INVALID_ARG || (accumulate != 0 && accumulate != 1)) return PT_ERR_INVALID_ARG;
    if (st) return st;
    if (M == 0 && accumulate) return PT_OK;
    if (!main_grad || (M > 0 && (!x || !dy))) return PT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(dy, 16) || !aligned(main_grad, 16) || !aligned(dbias, 16)) return PT_ERR_MISALIGNED;
    const LinearPlan plan = plan_of(PT_OP_WGRAD, M, N, K);
    const int64_t at = plan.partial_bytes, need = at + (dbias && M > 0 ? colsum_bytes(M, N) : 0);
    if (need && (!workspace || workspace_bytes < (size_t)need)) return PT_ERR_WORKSPACE;
    if (need && !aligned(workspace, 16)) return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    LinearParams p = {};
    p.a = (const uint16_t *)dy;
    p.b = (const uint16_t *)x;
    p.M = N;
    p.N = K;
    p.K = M;
    p.lda = N;
    p.ldb = K;
    p.partials = (float *)workspace;
    p.f.residual = accumulate ? main_grad : nullptr;
    p.f.out = main_grad;
    p.f.N = K;
    p.f.ldo = K;
    p.f.finish = kFinFwd;
    p.f.act = kActNone;
    p.f.f32 = 1;
    p.sums.dy = (const uint16_t *)dy;
    p.sums.dbias = dbias;
    p.sums.partials = (float *)((uint8_t *)workspace + at);
    p.sums.M = M;
    p.sums.N = N;
    p.sums.parts = colsum_parts(M, N);
    p.sums.accumulate = accumulate;
    return hip_status(launch_linear(p, kLinWgrad, plan, (hipStream_t)stream));
}

int pt_linear_act_bwd(const void *dout, const void *c, void *dc, int64_t M, int64_t N, int act, float swiglu_limit,
                      void *stream)
{
    const int st = check_product(M, N, 8);
    if (st == PT_ERR_INVALID_ARG || !is_act(act) || act == PT_ACT_NONE || swiglu_limit != swiglu_limit)
        return PT_ERR_INVALID_ARG;
    if (st) return st;
    if (act == PT_ACT_SWIGLU && N % 16) return PT_ERR_UNSUPPORTED;
    if (M == 0) return PT_OK;
    if (!dout || !c || !dc) return PT_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(c, 16) || !aligned(dc, 16)) return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    return hip_status(launch_act_bwd((const uint16_t *)dout, (const uint16_t *)c, (uint16_t *)dc, M, N, act,
                                     glu_limit(swiglu_limit), (hipStream_t)stream));
}

size_t pt_block_norm_workspace_size(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || rows > kMaxRows || cols > kBlockMaxCols) return 0;
    return (size_t)block_norm_parts(rows, cols) * 2 * (size_t)cols * 4;
}

int pt_block_norm_fwd(const void *x, const void *residual, const void *post_weight, const void *gate,
                      const void *pre_weight, void *residual_out, void *y, void *q, void *scales, float *rstd_post,
                      float *rstd_pre, int64_t rows, int64_t cols, float eps, float branch_scale, float residual_scale,
                      int gate_kind, int stream_dtype, int code_dtype, void *stream)
{
    const int st = check_block_norm(rows, cols, branch_scale, residual_scale, gate_kind, stream_dtype);
    if (st == PT_ERR_INVALID_ARG || !(eps >= 0.0f)) return PT_ERR_INVALID_ARG;
    if (st) return st;
    if (code_dtype != PT_BF16 && code_dtype != PT_MXFP8_E4M3 && code_dtype != PT_FP8_E4M3_ROWWISE)
        return PT_ERR_UNSUPPORTED;
    if (code_dtype == PT_MXFP8_E4M3 && cols % 32) return PT_ERR_UNSUPPORTED;
    if (rows == 0) return PT_OK;
    const bool codes = code_dtype != PT_BF16;
    if (!x || !residual || !residual_out || (gate != nullptr) != (gate_kind != PT_BLOCK_GATE_NONE)) return PT_ERR_INVALID_ARG;
    if (codes ? !q || !scales : q || scales) return PT_ERR_INVALID_ARG;
    // the next block's operand exists where its norm does
    if (pre_weight ? !y && !codes : y || codes || rstd_pre) return PT_ERR_INVALID_ARG;
    if (!post_weight && rstd_post) return PT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(post_weight, 16) || !aligned(pre_weight, 16) ||
        !aligned(residual_out, 16) || !aligned(y, 16) || !aligned(q, 16) || !aligned(rstd_post, 4) || !aligned(rstd_pre, 4) ||
        !aligned(gate, gate_kind == PT_BLOCK_GATE_ROWS ? 4 : 16) || (code_dtype == PT_FP8_E4M3_ROWWISE && !aligned(scales, 4)))
        return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    BlockNormFwdParams p = {};
    p.x = (const uint16_t *)x;
    p.residual = residual;
    p.post = (const uint16_t *)post_weight;
    p.gate = gate;
    p.pre = (const uint16_t *)pre_weight;
    p.residual_out = residual_out;
    p.y = (uint16_t *)y;
    p.q = (uint8_t *)q;
    p.scales = scales;
    p.rstd_post = rstd_post;
    p.rstd_pre = rstd_pre;
    p.rows = rows;
    p.cols = (int)cols;
    p.eps = eps;
    p.branch_scale = branch_scale;
    p.residual_scale = residual_scale;
    p.gate_kind = gate_kind;
    p.f32 = stream_dtype == PT_FP32;
    p.codes = code_dtype == PT_MXFP8_E4M3 ? kCodesMx : codes ? kCodesRows : kCodesNone;
    return hip_status(launch_block_norm_fwd(p, (hipStream_t)stream));
}

int pt_block_norm_bwd(const void *dy, const void *dres, const void *x, const void *s, const void *post_weight,
                      const void *gate, const void *pre_weight, const float *rstd_post, const float *rstd_pre, void *dx,
                      void *dresidual, void *dgate, float *dpost, float *dpre, int64_t rows, int64_t cols,
                      float branch_scale, float residual_scale, int gate_kind, int stream_dtype, int accumulate,
                      void *workspace, size_t workspace_bytes, void *stream)
{
    const int st = check_block_norm(rows, cols, branch_scale, residual_scale, gate_kind, stream_dtype);
    if (st == PT_ERR_INVALID_ARG || (accumulate != 0 && accumulate != 1)) return PT_ERR_INVALID_ARG;
    if (st) return st;
    if ((dpost && !post_weight) || (dpre && !pre_weight) || (dgate && gate_kind == PT_BLOCK_GATE_NONE)) return PT_ERR_INVALID_ARG;
    // sums over rows: they are written also where there are no rows
    const bool sums = dpost || dpre || (dgate && gate_kind == PT_BLOCK_GATE_COLS);
    if (rows == 0 && (!sums || accumulate)) return PT_OK;
    // the sums' last step reads the gate whatever the rows are
    if ((gate != nullptr) != (gate_kind != PT_BLOCK_GATE_NONE)) return PT_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!x || !dx || !dresidual) return PT_ERR_INVALID_ARG;
        if (pre_weight ? !dy || !s || !rstd_pre : dy != nullptr) return PT_ERR_INVALID_ARG;
        if (!pre_weight && !dres) return PT_ERR_INVALID_ARG;        // no gradient comes in at all
        if (post_weight && !rstd_post) return PT_ERR_INVALID_ARG;
    }
    const bool gate_sum = gate_kind == PT_BLOCK_GATE_ROWS;
    if (!aligned(dy, 16) || !aligned(dres, 16) || !aligned(x, 16) || !aligned(s, 16) || !aligned(post_weight, 16) ||
        !aligned(pre_weight, 16) || !aligned(gate, gate_sum ? 4 : 16) || !aligned(dgate, gate_sum ? 4 : 16) ||
        !aligned(rstd_post, 4) || !aligned(rstd_pre, 4) || !aligned(dx, 16) || !aligned(dresidual, 16) ||
        !aligned(dpost, 16) || !aligned(dpre, 16))
        return PT_ERR_MISALIGNED;
    if (sums && rows > 0) {
        if (!workspace || workspace_bytes < pt_block_norm_workspace_size(rows, cols)) return PT_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return PT_ERR_MISALIGNED;
    }
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    BlockNormBwdParams p = {};
    p.dy = (const uint16_t *)dy;
    p.dres = dres;
    p.x = (const uint16_t *)x;
    p.s = s;
    p.post = (const uint16_t *)post_weight;
    p.gate = gate;
    p.pre = (const uint16_t *)pre_weight;
    p.rstd_post = rstd_post;
    p.rstd_pre = rstd_pre;
    p.dx = (uint16_t *)dx;
    p.dresidual = dresidual;
    p.dgate = dgate;
    p.dpost = dpost;
    p.dpre = dpre;
    p.partials = sums ? (float *)workspace : nullptr;
    p.rows = rows;
    p.cols = (int)cols;
    p.branch_scale = branch_scale;
    p.residual_scale = residual_scale;
    p.gate_kind = gate_kind;
    p.f32 = stream_dtype == PT_FP32;
    p.accumulate = accumulate;
    p.sums = sums;
    return hip_status(launch_block_norm_bwd(p, (hipStream_t)stream));
}

int pt_moe_combine(const void *rows, const float *weights, const int32_t *row_of, const void *base, void *out, int64_t T,
                   int64_t M, int64_t H, int64_t k, void *stream)
{
    const int st = check_combine(T, M, H, k);
    if (st) return st;
    if (T == 0) return PT_OK;
    if ((M > 0 && !rows) || !row_of || !out) return PT_ERR_INVALID_ARG;
    if (!aligned(rows, 16) || !aligned(weights, 4) || !aligned(row_of, 4) || !aligned(base, 16) || !aligned(out, 16))
        return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    CombineParams p = {};
    p.rows = (const uint16_t *)rows;
    p.weights = weights;
    p.row_of = row_of;
    p.base = (const uint16_t *)base;
    p.out = (uint16_t *)out;
    p.T = T;
    p.M = M;
    p.H = (int)H;
    p.k = (int)k;
    return hip_status(launch_combine(p, (hipStream_t)stream));
}

int pt_moe_combine_bwd(const void *dout, const void *rows, const float *weights, const int32_t *row_of, void *drows,
                       float *dweights, int64_t T, int64_t M, int64_t H, int64_t k, void *stream)
{
    const int st = check_combine(T, M, H, k);
    if (st) return st;
    if (T == 0) return PT_OK;
    if (!dout || !row_of || (!drows && !dweights) || (dweights && M > 0 && !rows)) return PT_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(rows, 16) || !aligned(weights, 4) || !aligned(row_of, 4) || !aligned(drows, 16) ||
        !aligned(dweights, 4))
        return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    CombineBwdParams p = {};
    p.dout = (const uint16_t *)dout;
    p.rows = (const uint16_t *)rows;
    p.weights = weights;
    p.row_of = row_of;
    p.drows = (uint16_t *)drows;
    p.dweights = dweights;
    p.T = T;
    p.M = M;
    p.H = (int)H;
    p.k = (int)k;
    return hip_status(launch_combine_bwd(p, (hipStream_t)stream));
}

}  // extern "C"
