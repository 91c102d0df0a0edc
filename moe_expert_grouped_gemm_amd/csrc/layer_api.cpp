// layer_api.cpp -- the C ABI (include/ptgg.h) of the operators around the
// expert GEMM: residual RMS norm, router, whole layer for a few tokens.
// Argument checks and dispatch; nothing here reads device memory, allocates
// or synchronises.
#include "checks.hpp"
#include "layer.hpp"

using namespace ptgg;

namespace {

constexpr int64_t kWsHead = 256;                   // the error word

int check_gate(int logits_dtype, int gate, int renorm, float scale)
{
    if (gate != PT_GATE_SOFTMAX && gate != PT_GATE_SIGMOID) return PT_ERR_INVALID_ARG;
    if (renorm != 0 && renorm != 1) return PT_ERR_INVALID_ARG;
    if (scale != scale) return PT_ERR_INVALID_ARG;
    if (logits_dtype != PT_FP32 && logits_dtype != PT_BF16) return PT_ERR_UNSUPPORTED;
    return PT_OK;
}

int check_choice(int64_t T, int64_t E, int64_t k)
{
    if (T < 0 || E < 1 || k < 1 || k > E) return PT_ERR_INVALID_ARG;
    if (E > PT_MAX_GROUPS || k > PT_MAX_TOPK || T > kMaxRows) return PT_ERR_UNSUPPORTED;
    return PT_OK;
}

int64_t route_bytes(int64_t T, int64_t E) { return kWsHead + (T > kRouteChunk ? round256((int64_t)route_parts(T) * route_pitch((int)E) * 2) : 0); }

// The few-token layer's workspace, in bytes from its start.
struct FewWs {
    int64_t lens, row_of, token_of, plan, h, y, total;
};
FewWs few_ws(int64_t T, int64_t E, int64_t H, int64_t I, int64_t k)
{
    FewWs w;
    w.lens = kWsHead;
    w.row_of = w.lens + round256(E * 8);
    w.token_of = w.row_of + round256(T * k * 4);
    w.plan = w.token_of + round256(T * k * 4);
    w.h = w.plan + round256(16 + (int64_t)sizeof(FewBlock) * T * k);
    w.y = w.h + round256(T * k * I * 2);
    w.total = w.y + round256(T * k * H * 4);
    return w;
}

}  // namespace

extern "C" {

size_t pt_rmsnorm_workspace_size(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || rows > kMaxRows || cols > kNormMaxCols) return 0;
    const int parts = norm_bwd_parts(rows);
    return parts > 1 ? (size_t)parts * (size_t)cols * 4 : 0;
}

int pt_rmsnorm_fwd(const void *x, const void *residual, const void *weight, void *residual_out, void *y, void *q,
                   void *scales, float *rstd, int64_t rows, int64_t cols, float eps, int stream_dtype, int code_dtype,
                   void *stream)
{
    if (rows < 0 || cols < 1 || !(eps >= 0.0f)) return PT_ERR_INVALID_ARG;
    if (stream_dtype != PT_BF16 && stream_dtype != PT_FP32) return PT_ERR_UNSUPPORTED;
    if (code_dtype != PT_BF16 && code_dtype != PT_MXFP8_E4M3 && code_dtype != PT_FP8_E4M3_ROWWISE)
        return PT_ERR_UNSUPPORTED;
    const bool codes = code_dtype != PT_BF16;
    if (cols % 8 || (code_dtype == PT_MXFP8_E4M3 && cols % 32)) return PT_ERR_UNSUPPORTED;
    if (cols > kNormMaxCols || rows > kMaxRows) return PT_ERR_UNSUPPORTED;
    if (rows == 0) return PT_OK;
    if (!x || !weight || (residual && !residual_out) || (codes && (!q || !scales)) || (!codes && (q || scales)) ||
        (!y && !codes))
        return PT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
        !aligned(y, 16) || !aligned(q, 16) || !aligned(rstd, 4) ||
        (code_dtype == PT_FP8_E4M3_ROWWISE && !aligned(scales, 4)))
        return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    NormFwdParams p = {};
    p.x = (const uint16_t *)x;
    p.residual = residual;
    p.weight = (const uint16_t *)weight;
    p.residual_out = residual_out;
    p.y = (uint16_t *)y;
    p.q = (uint8_t *)q;
    p.scales = scales;
    p.rstd = rstd;
    p.rows = rows;
    p.cols = (int)cols;
    p.eps = eps;
    p.f32 = stream_dtype == PT_FP32;
    p.codes = code_dtype == PT_MXFP8_E4M3 ? kCodesMx : codes ? kCodesRows : kCodesNone;
    return hip_status(launch_rmsnorm_fwd(p, (hipStream_t)stream));
}

int pt_rmsnorm_bwd(const void *dy, const void *s, const void *weight, const float *rstd, const void *dres, void *ds,
                   float *dweight, int64_t rows, int64_t cols, int stream_dtype, int accumulate, void *workspace,
                   size_t workspace_bytes, void *stream)
{
    if (rows < 0 || cols < 1 || (accumulate != 0 && accumulate != 1)) return PT_ERR_INVALID_ARG;
    if (stream_dtype != PT_BF16 && stream_dtype != PT_FP32) return PT_ERR_UNSUPPORTED;
    if (cols % 8 || cols > kNormMaxCols || rows > kMaxRows) return PT_ERR_UNSUPPORTED;
    if (rows == 0 && (!dweight || accumulate)) return PT_OK;
    if (rows > 0 && (!dy || !s || !weight || !rstd || !ds)) return PT_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(s, 16) || !aligned(weight, 16) || !aligned(rstd, 4) || !aligned(dres, 16) ||
        !aligned(ds, 16) || !aligned(dweight, 16))
        return PT_ERR_MISALIGNED;
    const size_t need = dweight ? pt_rmsnorm_workspace_size(rows, cols) : 0;
    if (need && (!workspace || workspace_bytes < need)) return PT_ERR_WORKSPACE;
    if (need && !aligned(workspace, 16)) return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    NormBwdParams p = {};
    p.dy = (const uint16_t *)dy;
    p.s = s;
    p.weight = (const uint16_t *)weight;
    p.rstd = rstd;
    p.dres = dres;
    p.ds = ds;
    p.dweight = dweight;
    p.partials = (float *)workspace;
    p.rows = rows;
    p.cols = (int)cols;
    p.f32 = stream_dtype == PT_FP32;
    p.accumulate = accumulate;
    return hip_status(launch_rmsnorm_bwd(p, (hipStream_t)stream));
}

size_t pt_moe_route_workspace_size(int64_t T, int64_t E, int64_t k)
{
    return check_choice(T, E, k) == PT_OK ? (size_t)route_bytes(T, E) : 0;
}

int pt_moe_route(const void *logits, const float *bias, int32_t *topk_ids, float *topk_weights, int64_t *lens,
                 int32_t *row_of, int32_t *token_of, int64_t T, int64_t E, int64_t k, int logits_dtype, int gate,
                 int renorm, float scale, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = check_choice(T, E, k);
    if (!st) st = check_gate(logits_dtype, gate, renorm, scale);
    if (st) return st;
    if (bias && gate != PT_GATE_SIGMOID) return PT_ERR_INVALID_ARG;
    if (!lens || (T > 0 && (!logits || !topk_ids || !topk_weights || !row_of || !token_of))) return PT_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(bias, 16) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
        !aligned(lens, 8) || !aligned(row_of, 4) || !aligned(token_of, 4) || !aligned(workspace, 16))
        return PT_ERR_MISALIGNED;
    if (T > kRouteChunk && (!workspace || workspace_bytes < (size_t)route_bytes(T, E))) return PT_ERR_WORKSPACE;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    RouteParams p = {};
    p.logits = logits;
    p.bias = bias;
    p.topk_ids = topk_ids;
    p.topk_weights = topk_weights;
    p.lens = lens;
    p.row_of = row_of;
    p.token_of = token_of;
    p.counts = (uint16_t *)((uint8_t *)workspace + kWsHead);
    p.err = workspace && workspace_bytes >= 4 ? (uint32_t *)workspace : nullptr;
    p.T = T;
    p.E = (int)E;
    p.k = (int)k;
    p.bf16 = logits_dtype == PT_BF16;
    p.sigmoid = gate == PT_GATE_SIGMOID;
    p.renorm = renorm;
    p.scale = scale;
    return hip_status(launch_moe_route(p, (hipStream_t)stream));
}

int pt_moe_route_bwd(const void *logits, const int32_t *topk_ids, const float *dweights, void *dlogits, int64_t T,
                     int64_t E, int64_t k, int logits_dtype, int gate, int renorm, float scale, void *stream)
{
    int st = check_choice(T, E, k);
    if (!st) st = check_gate(logits_dtype, gate, renorm, scale);
    if (st) return st;
    if (T == 0) return PT_OK;
    if (!logits || !topk_ids || !dweights || !dlogits) return PT_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(dlogits, 16) || !aligned(topk_ids, 4) || !aligned(dweights, 4))
        return PT_ERR_MISALIGNED;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    RouteBwdParams p = {};
    p.logits = logits;
    p.topk_ids = topk_ids;
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.T = T;
    p.E = (int)E;
    p.k = (int)k;
    p.bf16 = logits_dtype == PT_BF16;
    p.sigmoid = gate == PT_GATE_SIGMOID;
    p.renorm = renorm;
    p.scale = scale;
    return hip_status(launch_moe_route_bwd(p, (hipStream_t)stream));
}

size_t pt_moe_few_tokens_workspace_size(int64_t T, int64_t E, int64_t H, int64_t I, int64_t k)
{
    if (check_choice(T, E, k) != PT_OK || T > kFewMaxTokens || H < 1 || I < 1 || H > kFewMaxWidth || I > kFewMaxWidth)
        return 0;
    return (size_t)few_ws(T, E, H, I, k).total;
}

int pt_moe_few_tokens(const void *x, const void *logits, const float *bias, const void *w1, const uint8_t *w1_scale,
                      const void *w2, const uint8_t *w2_scale, void *out, int32_t *topk_ids, float *topk_weights,
                      int64_t T, int64_t E, int64_t H, int64_t I, int64_t k, int logits_dtype, int gate, int renorm,
                      float scale, int weight_dtype, float swiglu_limit, void *workspace, size_t workspace_bytes,
                      void *stream)
{
    int st = check_choice(T, E, k);
    if (!st) st = check_gate(logits_dtype, gate, renorm, scale);
    if (st) return st;
    if (H < 1 || I < 1 || swiglu_limit != swiglu_limit) return PT_ERR_INVALID_ARG;
    if (bias && gate != PT_GATE_SIGMOID) return PT_ERR_INVALID_ARG;
    if (weight_dtype != PT_BF16 && weight_dtype != PT_MXFP8_E4M3 && weight_dtype != PT_MXFP4_E2M1)
        return PT_ERR_UNSUPPORTED;
    const bool mx = weight_dtype != PT_BF16;
    const int64_t grain = mx ? 32 : 8;
    if (T > kFewMaxTokens || H % grain || I % grain || H > kFewMaxWidth || I > kFewMaxWidth) return PT_ERR_UNSUPPORTED;
    if (T == 0) return PT_OK;
    if (!x || !logits || !w1 || !w2 || !out || !topk_ids || !topk_weights) return PT_ERR_INVALID_ARG;
    if ((w1_scale != nullptr) != mx || (w2_scale != nullptr) != mx) return PT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(logits, 16) || !aligned(bias, 16) || !aligned(w1, 16) || !aligned(w2, 16) ||
        !aligned(out, 16) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(workspace, 16))
        return PT_ERR_MISALIGNED;
    const FewWs w = few_ws(T, E, H, I, k);
    if (!workspace || workspace_bytes < (size_t)w.total) return PT_ERR_WORKSPACE;
    if (!device_is_gfx950()) return PT_ERR_UNSUPPORTED;
    uint8_t *ws = (uint8_t *)workspace;
    FewParams p = {};
    p.x = (const uint16_t *)x;
    p.w1 = (const uint8_t *)w1;
    p.w1s = w1_scale;
    p.w2 = (const uint8_t *)w2;
    p.w2s = w2_scale;
    p.out = (uint16_t *)out;
    p.route.logits = logits;
    p.route.bias = bias;
    p.route.topk_ids = topk_ids;
    p.route.topk_weights = topk_weights;
    p.route.lens = (int64_t *)(ws + w.lens);
    p.route.row_of = (int32_t *)(ws + w.row_of);
    p.route.token_of = (int32_t *)(ws + w.token_of);
    p.route.err = (uint32_t *)ws;
    p.route.T = T;
    p.route.E = (int)E;
    p.route.k = (int)k;
    p.route.bf16 = logits_dtype == PT_BF16;
    p.route.sigmoid = gate == PT_GATE_SIGMOID;
    p.route.renorm = renorm;
    p.route.scale = scale;
    p.plan = (int *)(ws + w.plan);
    p.h = (uint16_t *)(ws + w.h);
    p.y = (float *)(ws + w.y);
    p.T = (int)T;
    p.E = (int)E;
    p.H = (int)H;
    p.I = (int)I;
    p.k = (int)k;
    p.weights = weight_dtype == PT_MXFP8_E4M3 ? kFewMxfp8 : mx ? kFewMxfp4 : kFewBf16;
    const float inf = __builtin_huge_valf();
    p.swiglu_limit = swiglu_limit > 0.0f && swiglu_limit < inf ? swiglu_limit : inf;
    return hip_status(launch_few_tokens(p, (hipStream_t)stream));
}

}  // extern "C"
