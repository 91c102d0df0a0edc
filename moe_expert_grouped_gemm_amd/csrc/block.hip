// block.hip -- what surrounds a block's products: the norms after and before a
// block with its gate and residual scale, and the weighted sum that brings the
// experts' rows back to their tokens; forward and backward.
//
// Norms forward, per row, with a = branch_scale, b = residual_scale:
//     u = x rpost wpost,  h = b residual + a gate u,  v = h rpre wpre,
//     rpost = (mean(x^2) + eps)^-1/2,  rpre = (mean(h^2) + eps)^-1/2
// h is rounded once to the stream's type, and rpre is that of the rounded
// stream; v leaves in bf16 and as E4M3 codes of the unrounded value.
//
// Backward, per row, with hh = h rpre, xh = x rpost, g = dy wpre:
//     ds = dres + rpre (g - hh mean(g hh)),           dresidual = b ds
//     t = a ds xh,  du = a gate ds,  e = du wpost,    dx = rpost (e - xh mean(e xh))
//     dwpre = sum dy hh,  dwpost = sum gate t,        dgate = t wpost, summed to its shape
// A gate per column is the same in every row, so that sum t serves its gradient
// and wpost's alike.
//
// All are bound by memory: each element is read and written once, the row
// staying in registers between its sums and its outputs.
#include "dense.hpp"
#include "layer.hpp"
#include "rows.hpp"

namespace ptgg {

namespace {

// Traffic from which a call's rows go past the caches.
constexpr int64_t kBlockStreamBytes = (int64_t)80 << 20;

__host__ __device__ constexpr int team_threads(int W) { return W > 1 ? 64 * W : kThreads; }

// The gate's bf16 values of row r (element base of the matrix), or null where it
// is one number a row.  One address for both layouts, chosen once per row and before
// the loop over the row's columns: with a load for each layout inside the loop the
// compiler joined the two into one that took the whole matrix's address for a gate
// per column as well, far past the vector's end.
__device__ __forceinline__ const uint16_t *gate_row(const void *gate, int kind, int64_t base)
{
    return kind == kGateCols || kind == kGateFull ? (const uint16_t *)gate + (kind == kGateFull ? base : 0) : nullptr;
}
__device__ __forceinline__ void gate8(const uint16_t *row, int e, float row_gate, float (&f)[8])
{
    if (row) unpack8(*(const uintx4 *)(row + e), f);
    else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = row_gate;
    }
}

// W waves hold one row, NV groups of 8 values per lane.
template <bool F32, int CODES, int W, int NV, bool NT>
__global__ __launch_bounds__(team_threads(W)) void block_norm_fwd_kernel(BlockNormFwdParams p)
{
    constexpr int TEAM = 64 * W, ROWS = team_threads(W) / TEAM;
    __shared__ float s_post[W], s_pre[W];
    __shared__ uint32_t s_max[W];
    const int t = (int)threadIdx.x % TEAM;
    const int64_t r = (int64_t)blockIdx.x * ROWS + (int)threadIdx.x / TEAM;
    if (r >= p.rows) return;                 // whole teams: W > 1 has one row per workgroup
    const int n8 = p.cols >> 3;
    const int64_t base = r * p.cols;
    uintx4 xv[NV];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = i * TEAM + t;
        xv[i] = uintx4{0, 0, 0, 0};
        if (g < n8) xv[i] = load_as<NT, uintx4>(p.x + base + g * 8);
    }
    // the residual's loads go out before the first sum is waited for
    float h[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = i * TEAM + t;
        if (g < n8) load_stream<F32, NT>(p.residual, base + g * 8, h[i]);
        else {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
        }
    }
    float rpost = 1.0f;
    if (p.post) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float x[8];
            unpack8(xv[i], x);
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) part = __builtin_fmaf(x[j], x[j], part);
            sq += part;
        }
        sq = team_sum<W>(sq, s_post);
        rpost = 1.0f / __builtin_sqrtf(sq / (float)p.cols + p.eps);
        if (t == 0 && p.rstd_post) p.rstd_post[r] = rpost;
    }
    const float row_gate = p.gate_kind == kGateRows ? ((const float *)p.gate)[r] : 1.0f;
    const uint16_t *gates = gate_row(p.gate, p.gate_kind, base);
    sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = i * TEAM + t;
        if (g < n8) {
            float x[8], k[8];
            unpack8(xv[i], x);
            gate8(gates, g * 8, row_gate, k);
            if (p.post) {
                float w[8];
                unpack8(*(const uintx4 *)(p.post + g * 8), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * rpost * w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = __builtin_fmaf(p.branch_scale * k[j], x[j], p.residual_scale * h[i][j]);
            if constexpr (!F32) {
                const uintx4 b = pack8(h[i]);
                store_as<NT>((uint16_t *)p.residual_out + base + g * 8, b);
                unpack8(b, h[i]);
            } else {
                store_stream<true, NT>(p.residual_out, base + g * 8, h[i]);
            }
        }
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) part = __builtin_fmaf(h[i][j], h[i][j], part);
        sq += part;
    }
    if (!p.pre) return;
    sq = team_sum<W>(sq, s_pre);
    const float rpre = 1.0f / __builtin_sqrtf(sq / (float)p.cols + p.eps);
    if (t == 0 && p.rstd_pre) p.rstd_pre[r] = rpre;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = i * TEAM + t;
        if (g < n8) {
            float w[8];
            unpack8(*(const uintx4 *)(p.pre + g * 8), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * rpre * w[j];
            if (p.y) store_as<NT>(p.y + base + g * 8, pack8(h[i]));
            if constexpr (CODES == kCodesMx) {
                const uint32_t E = mx_scale_byte<8>(quad_max_u32(amax8(h[i])) >> 16);
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = __builtin_ldexpf(h[i][j], 127 - (int)E);
                *(uintx2 *)(p.q + base + g * 8) = codes8(f);
                if ((t & 3) == 0) ((uint8_t *)p.scales)[(base >> 5) + (g >> 2)] = (uint8_t)E;
            }
            if constexpr (CODES == kCodesRows) amax = max(amax, amax8(h[i]));
        }
    }
    if constexpr (CODES == kCodesRows) {
        const float mf = bits_f32(team_max_u32<W>(amax, s_max));
        const float f = mf == 0.0f ? 1.0f : __builtin_fminf(448.0f / mf, 3.40282346638528859812e+38f);
        const float scale = mf != mf ? mf : f;       // fminf would turn a NaN factor into a number
        if (t == 0) ((float *)p.scales)[r] = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int g = i * TEAM + t;
            if (g < n8) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = h[i][j] * scale;
                *(uintx2 *)(p.q + base + g * 8) = codes8(v);
            }
        }
    }
}

template <bool F32, int CODES, bool NT>
void launch_fwd_as(const BlockNormFwdParams &p, hipStream_t s)
{
    const int n8 = p.cols / 8;
#define PTGG_NORM(W, NV)                                                                                       \
    hipLaunchKernelGGL((block_norm_fwd_kernel<F32, CODES, W, NV, NT>),                                         \
                       dim3((unsigned)((p.rows + team_threads(W) / 64 / W - 1) / (team_threads(W) / 64 / W))), \
                       dim3(team_threads(W)), 0, s, p)
    if (n8 <= 64) PTGG_NORM(1, 1);
    else if (n8 <= 128) PTGG_NORM(1, 2);
    else if (n8 <= 256) PTGG_NORM(4, 1);
    else if (n8 <= 512) PTGG_NORM(4, 2);
    else if (n8 <= 768) PTGG_NORM(4, 3);
    else if (n8 <= 1024) PTGG_NORM(4, 4);
    else PTGG_NORM(8, 4);
#undef PTGG_NORM
}

template <bool F32, int CODES>
hipError_t launch_fwd(const BlockNormFwdParams &p, hipStream_t s)
{
    const int64_t bytes = p.rows * p.cols * (F32 ? 12 : 8);
    if (bytes > kBlockStreamBytes) launch_fwd_as<F32, CODES, true>(p, s);
    else launch_fwd_as<F32, CODES, false>(p, s);
    return hipGetLastError();
}

// ------------------------------------------------------------------ norms backward
// What the call has, known when the kernel is compiled where it is all there: a
// branch on each operand costs registers that the rows in flight need (16384 x 2880
// with a gate per channel: 146 us, 129 without them).
template <int GATE>
struct Has {
    static constexpr bool ALL = GATE >= 0;
    const BlockNormBwdParams &p;
    __device__ __forceinline__ bool pre() const { return ALL || p.pre; }
    __device__ __forceinline__ bool post() const { return ALL || p.post; }
    __device__ __forceinline__ bool dres() const { return ALL || p.dres; }
    __device__ __forceinline__ int gate() const { return ALL ? GATE : p.gate_kind; }
};

// The loads of a row's share as they come, so that the next rows' can be in
// flight while this one is worked on.
template <bool F32, int GATE, int TEAM, int NV, bool NT>
struct BlockRow {
    static constexpr int SV = F32 ? 2 : 1;               // 16-byte loads per 8 stream values
    static constexpr bool MAY_FULL = GATE < 0 || GATE == kGateFull;
    uintx4 dy[NV], x[NV], gate[MAY_FULL ? NV : 1], s[NV * SV], dres[NV * SV];
    float rpost, rpre, row_gate;
    __device__ __forceinline__ void load(const BlockNormBwdParams &p, int64_t r, int t)
    {
        const Has<GATE> has{p};
        const int64_t base = r * p.cols;
        rpost = has.post() ? p.rstd_post[r] : 1.0f;
        rpre = has.pre() ? p.rstd_pre[r] : 1.0f;
        row_gate = has.gate() == kGateRows ? ((const float *)p.gate)[r] : 1.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TEAM + t) * 8;
            if (e < p.cols) {
                const int64_t at = (base + e) * (F32 ? 4 : 2);
                x[i] = load_as<NT, uintx4>(p.x + base + e);
                if (has.pre()) {
                    dy[i] = load_as<NT, uintx4>(p.dy + base + e);
#pragma unroll
                    for (int j = 0; j < SV; ++j) s[i * SV + j] = load_as<NT && !F32, uintx4>((const uint8_t *)p.s + at + 16 * j);
                }
                if (has.dres()) {
#pragma unroll
                    for (int j = 0; j < SV; ++j) dres[i * SV + j] = load_as<NT && !F32, uintx4>((const uint8_t *)p.dres + at + 16 * j);
                }
                if (MAY_FULL && has.gate() == kGateFull) gate[MAY_FULL ? i : 0] = load_as<NT, uintx4>((const uint16_t *)p.gate + base + e);
            }
        }
    }
    static __device__ __forceinline__ void widen(const uintx4 *v, float (&f)[8])
    {
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = bits_f32(v[0][j]), f[4 + j] = bits_f32(v[SV - 1][j]);
        } else {
            unpack8(v[0], f);
        }
    }
};

// W waves hold a row; a workgroup's teams take rows a grid apart and keep their
// lanes' two sums over rows in registers: a = dwpre, b = dwpost, or for a gate
// per column sum t.  The teams' are added in order, the workgroups' by
// block_norm_join_kernel.  The loads of the next two rows are in flight while one
// is worked on.
template <bool F32, int GATE, int W, int NV, bool NT>
__global__ __launch_bounds__(team_threads(W)) void block_norm_bwd_kernel(BlockNormBwdParams p, int parts)
{
    constexpr int TEAM = 64 * W, TEAMS = team_threads(W) / TEAM;
    __shared__ float s_sum[6][W];
    __shared__ floatx4 s_acc[TEAMS > 1 ? (TEAMS - 1) * TEAM * NV * 4 : 1];
    const Has<GATE> has{p};
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    float a[NV][8] = {}, b[NV][8] = {};
    int flip = 0;
    const uint16_t *col_gate = has.gate() == kGateCols ? (const uint16_t *)p.gate : nullptr;
    const int64_t first = (int64_t)blockIdx.x * TEAMS + team, step = (int64_t)parts * TEAMS;
    using Row = BlockRow<F32, GATE, TEAM, NV, NT>;
    constexpr int AHEAD = NV > 1 || GATE < 0 ? 0 : F32 || GATE == kGateFull ? 1 : 2;     // what the registers hold
    auto work = [&](const Row &row, int64_t r) {
        const int64_t base = r * p.cols;
        float ds[NV][8];
        // ds = dres + rpre (g - h c)
        float c = 0.0f;
        if (has.pre()) {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * TEAM + t) * 8;
                if (e < p.cols) {
                    float h[8], w[8], g[8];
                    unpack8(row.dy[i], g);
                    row.widen(row.s + i * row.SV, h);
                    unpack8(*(const uintx4 *)(p.pre + e), w);
                    float part = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        a[i][j] = __builtin_fmaf(g[j], h[j] * row.rpre, a[i][j]);
                        ds[i][j] = g[j] * w[j];
                        part = __builtin_fmaf(ds[i][j], h[j], part);
                    }
                    dot += part;
                }
            }
            dot = team_sum<W>(dot, s_sum[flip]);
            c = row.rpre * row.rpre * (dot / (float)p.cols);
        }
        // dresidual, t, and e's product with x
        float dot = 0.0f, gsum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TEAM + t) * 8;
            if (e < p.cols) {
                float x[8], w[8], k[8], d[8] = {}, o[8], dg[8];
                if (has.dres()) row.widen(row.dres + i * row.SV, d);
                if (has.pre()) {
                    float h[8];
                    row.widen(row.s + i * row.SV, h);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] += row.rpre * (ds[i][j] - h[j] * c);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = p.residual_scale * d[j], d[j] *= p.branch_scale;
                store_stream<F32, NT>(p.dresidual, base + e, o);
                unpack8(row.x[i], x);
                if (Row::MAY_FULL && has.gate() == kGateFull) unpack8(row.gate[Row::MAY_FULL ? i : 0], k);
                else gate8(col_gate, e, row.row_gate, k);
                if (has.post()) unpack8(*(const uintx4 *)(p.post + e), w);
                else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = 1.0f;
                }
                float part = 0.0f, gpart = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float tt = d[j] * (x[j] * row.rpost);
                    b[i][j] += has.gate() == kGateCols ? tt : tt * k[j];
                    dg[j] = tt * w[j];
                    gpart += dg[j];
                    ds[i][j] = d[j] * k[j] * w[j];
                    part = __builtin_fmaf(ds[i][j], x[j], part);
                }
                if (has.gate() == kGateFull && p.dgate) store_as<NT>((uint16_t *)p.dgate + base + e, pack8(dg));
                dot += part;
                gsum += gpart;
            }
        }
        float c2 = 0.0f;
        if (has.post()) {
            dot = team_sum<W>(dot, s_sum[flip + 1]);
            c2 = row.rpost * row.rpost * (dot / (float)p.cols);
        }
        if (has.gate() == kGateRows && p.dgate) {
            gsum = team_sum<W>(gsum, s_sum[flip + 2]);
            if (t == 0) ((float *)p.dgate)[r] = gsum;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TEAM + t) * 8;
            if (e < p.cols) {
                float x[8], o[8];
                unpack8(row.x[i], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = row.rpost * (ds[i][j] - x[j] * c2);
                store_as<NT>(p.dx + base + e, pack8(o));
            }
        }
        flip ^= 3;                       // the next row's sums never meet readers of this one's
    };
    if constexpr (AHEAD == 0) {
        for (int64_t r = first; r < p.rows; r += step) {
            Row row;
            row.load(p, r, t);
            work(row, r);
        }
    } else {
        Row next[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (first + i * step < p.rows) next[i].load(p, first + i * step, t);
        for (int64_t r = first; r < p.rows; r += step) {
            const Row row = next[0];
            if (AHEAD > 1) next[0] = next[AHEAD - 1];
            if (r + AHEAD * step < p.rows) next[AHEAD - 1].load(p, r + AHEAD * step, t);
            work(row, r);
        }
    }
    if (!p.sums) return;
    if constexpr (TEAMS > 1) {
        if (team) {
            floatx4 *out = s_acc + (team - 1) * TEAM * NV * 4 + t;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                out[(4 * i) * TEAM] = floatx4{a[i][0], a[i][1], a[i][2], a[i][3]};
                out[(4 * i + 1) * TEAM] = floatx4{a[i][4], a[i][5], a[i][6], a[i][7]};
                out[(4 * i + 2) * TEAM] = floatx4{b[i][0], b[i][1], b[i][2], b[i][3]};
                out[(4 * i + 3) * TEAM] = floatx4{b[i][4], b[i][5], b[i][6], b[i][7]};
            }
        }
        __syncthreads();
        if (team) return;
#pragma unroll
        for (int k = 1; k < TEAMS; ++k) {
            const floatx4 *in = s_acc + (k - 1) * TEAM * NV * 4 + t;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    a[i][j] += in[(4 * i + j / 4) * TEAM][j & 3];
                    b[i][j] += in[(4 * i + 2 + j / 4) * TEAM][j & 3];
                }
        }
    }
    float *out = p.partials + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TEAM + t) * 8;
        if (e >= p.cols) continue;
        store_stream<true, false>(out, e, a[i]);
        store_stream<true, false>(out, p.cols + e, b[i]);
    }
}

// The parts' sums: dpre from a, and from b dpost, or of a gate per column dpost
// = gate b and dgate = wpost b.  A workgroup takes 32 columns of a and b: 8
// lanes of four, 128 rows of parts side by side, joined in LDS in their order.
constexpr int kJoinThreads = 1024, kJoinCols = 32;
__device__ __forceinline__ void put4(float *out, int c, floatx4 v, int accumulate)
{
    floatx4 *o = (floatx4 *)(out + c);
    *o = accumulate ? *o + v : v;
}
__device__ __forceinline__ floatx4 widen4(const uint16_t *p)
{
    const uintx2 v = *(const uintx2 *)p;
    return floatx4{bits_f32(v[0] << 16), bits_f32(v[0] & 0xFFFF0000u), bits_f32(v[1] << 16), bits_f32(v[1] & 0xFFFF0000u)};
}
__global__ __launch_bounds__(kJoinThreads) void block_norm_join_kernel(BlockNormBwdParams p, int parts)
{
    constexpr int SIDE = kJoinThreads / (kJoinCols / 4);
    __shared__ floatx4 s[SIDE][kJoinCols / 4 + 1];
    const int lane = threadIdx.x % (kJoinCols / 4), side = threadIdx.x / (kJoinCols / 4);
    const int c = (int)blockIdx.x * kJoinCols + lane * 4, which = blockIdx.y;
    floatx4 sum = {0, 0, 0, 0};
    if (c < p.cols) {
#pragma unroll 4
        for (int i = side; i < parts; i += SIDE) sum += *(const floatx4 *)(p.partials + ((int64_t)i * 2 + which) * p.cols + c);
    }
    s[side][lane] = sum;
    __syncthreads();
    for (int n = SIDE / 2; n >= 1; n /= 2) {
        if (side < n) s[side][lane] += s[side + n][lane];
        __syncthreads();
    }
    if (side || c >= p.cols) return;
    sum = s[0][lane];
    if (which == 0) {
        if (p.dpre) put4(p.dpre, c, sum, p.accumulate);
        return;
    }
    const bool cols = p.gate_kind == kGateCols;
    if (p.dpost) put4(p.dpost, c, cols ? sum * widen4((const uint16_t *)p.gate + c) : sum, p.accumulate);
    if (cols && p.dgate) put4((float *)p.dgate, c, p.post ? sum * widen4(p.post + c) : sum, p.accumulate);
}

// Waves of a row in the backward: 8 columns a lane, which leaves registers for the
// loads of two rows more (8192 x 4096 bf16: 90 us, 99 with 16 a lane and one row).
int bwd_waves(int64_t cols) { const int64_t n8 = cols / 8; return n8 <= 64 ? 1 : n8 <= 128 ? 2 : n8 <= 256 ? 4 : n8 <= 512 ? 8 : 16; }

template <bool F32, int GATE, bool NT>
void launch_bwd_rows(const BlockNormBwdParams &p, int parts, hipStream_t s)
{
#define PTGG_NORM(W, NV)                                                                                                   \
    hipLaunchKernelGGL((block_norm_bwd_kernel<F32, GATE, W, NV, NT>), dim3((unsigned)parts), dim3(team_threads(W)), 0, s, p, \
                       parts)
    switch (bwd_waves(p.cols)) {
    case 1: PTGG_NORM(1, 1); break;
    case 2: PTGG_NORM(2, 1); break;
    case 4: PTGG_NORM(4, 1); break;
    case 8: PTGG_NORM(8, 1); break;
    default:
        if (p.cols <= 8192) PTGG_NORM(16, 1);
        else PTGG_NORM(16, 2);
    }
#undef PTGG_NORM
}

template <bool F32, bool NT>
void launch_bwd_gate(const BlockNormBwdParams &p, int parts, hipStream_t s)
{
    if (!p.pre || !p.post || !p.dres) launch_bwd_rows<F32, -1, false>(p, parts, s);
    else if (p.gate_kind == kGateNone) launch_bwd_rows<F32, kGateNone, NT>(p, parts, s);
    else if (p.gate_kind == kGateCols) launch_bwd_rows<F32, kGateCols, NT>(p, parts, s);
    else if (p.gate_kind == kGateRows) launch_bwd_rows<F32, kGateRows, NT>(p, parts, s);
    else launch_bwd_rows<F32, kGateFull, NT>(p, parts, s);
}

template <bool F32>
hipError_t launch_bwd(const BlockNormBwdParams &p, hipStream_t s)
{
    const int parts = block_norm_parts(p.rows, p.cols);
    if (p.rows > 0) {
        const int64_t bytes = p.rows * p.cols * (F32 ? 18 : 12);
        if (bytes > kBlockStreamBytes) launch_bwd_gate<F32, true>(p, parts, s);
        else launch_bwd_gate<F32, false>(p, parts, s);
    }
    if (p.sums)
        hipLaunchKernelGGL(block_norm_join_kernel, dim3((unsigned)((p.cols + kJoinCols - 1) / kJoinCols), 2),
                           dim3(kJoinThreads), 0, s, p, p.rows > 0 ? parts : 0);
    return hipGetLastError();
}

// ------------------------------------------------------------------ experts' weighted sum
// A thread sums 8 columns of one token over its slots; the workgroup's threads
// take consecutive groups of 8 columns of consecutive tokens.
template <bool NT>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineParams p)
{
    const int n8 = p.H >> 3;
    const int64_t total = p.T * n8;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / n8;
        const int e = (int)(i - t * n8) * 8;
        float v[8] = {};
        if (p.base) unpack8(load_as<NT, uintx4>(p.base + t * p.H + e), v);
        for (int j0 = 0; j0 < p.k; j0 += 4) {
            uintx4 y[4];
            float w[4];
            bool ok[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t row = j0 + j < p.k ? p.row_of[t * p.k + j0 + j] : -1;
                ok[j] = row >= 0 && row < p.M;
                w[j] = p.weights && ok[j] ? p.weights[t * p.k + j0 + j] : 1.0f;
                if (ok[j]) y[j] = load_as<NT, uintx4>(p.rows + row * p.H + e);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!ok[j]) continue;
                float f[8];
                unpack8(y[j], f);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = __builtin_fmaf(w[j], f[c], v[c]);
            }
        }
        store_as<false>(p.out + t * p.H + e, pack8(v));
    }
}

// W waves hold a token's gradient, NV groups of 8 per lane, and go through its
// slots: the row's gradient out, its product with the row summed.
template <int W, int NV, bool NT>
__global__ __launch_bounds__(team_threads(W)) void combine_bwd_kernel(CombineBwdParams p)
{
    constexpr int TEAM = 64 * W, TEAMS = team_threads(W) / TEAM, KMAX = kRouteMaxTopk;
    __shared__ float s_dot[TEAMS][KMAX][W];
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    const int64_t tok = (int64_t)blockIdx.x * TEAMS + team;
    const bool live = tok < p.T;
    const int n8 = p.H >> 3;
    uintx4 d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = i * TEAM + t;
        d[i] = uintx4{0, 0, 0, 0};
        if (live && g < n8) d[i] = load_as<NT, uintx4>(p.dout + tok * p.H + g * 8);
    }
    if (live) {
        for (int j = 0; j < p.k; ++j) {
            const int64_t row = p.row_of[tok * p.k + j];
            const bool ok = row >= 0 && row < p.M;
            float dot = 0.0f;
            if (ok) {
                const float w = p.weights ? p.weights[tok * p.k + j] : 1.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int g = i * TEAM + t;
                    if (g < n8) {
                        float f[8], o[8];
                        unpack8(d[i], f);
                        if (p.dweights) {
                            float y[8], part = 0.0f;
                            unpack8(load_as<NT, uintx4>(p.rows + row * p.H + g * 8), y);
#pragma unroll
                            for (int c = 0; c < 8; ++c) part = __builtin_fmaf(f[c], y[c], part);
                            dot += part;
                        }
                        if (p.drows) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) o[c] = w * f[c];
                            store_as<NT>(p.drows + row * p.H + g * 8, pack8(o));
                        }
                    }
                }
            }
            if (p.dweights) {
                dot = wave_sum(dot);
                if ((threadIdx.x & 63) == 0) s_dot[team][j][t >> 6] = dot;
            }
        }
    }
    if (!p.dweights) return;
    __syncthreads();
    if (live && t < p.k) {
        float sum = s_dot[team][t][0];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += s_dot[team][t][w];
        p.dweights[tok * p.k + t] = sum;
    }
}

template <bool NT>
hipError_t launch_combine_bwd_as(const CombineBwdParams &p, hipStream_t s)
{
    const int n8 = p.H / 8;
#define PTGG_COMBINE(W, NV)                                                                                     \
    hipLaunchKernelGGL((combine_bwd_kernel<W, NV, NT>),                                                         \
                       dim3((unsigned)((p.T + team_threads(W) / 64 / W - 1) / (team_threads(W) / 64 / W))),      \
                       dim3(team_threads(W)), 0, s, p)
    if (n8 <= 64) PTGG_COMBINE(1, 1);
    else if (n8 <= 128) PTGG_COMBINE(1, 2);
    else if (n8 <= 256) PTGG_COMBINE(4, 1);
    else if (n8 <= 512) PTGG_COMBINE(4, 2);
    else if (n8 <= 1024) PTGG_COMBINE(4, 4);
    else if (n8 <= 2048) PTGG_COMBINE(8, 4);
    else PTGG_COMBINE(8, 8);
#undef PTGG_COMBINE
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNormFwdParams &p, hipStream_t s)
{
    switch (p.codes) {
    case kCodesMx: return p.f32 ? launch_fwd<true, kCodesMx>(p, s) : launch_fwd<false, kCodesMx>(p, s);
    case kCodesRows: return p.f32 ? launch_fwd<true, kCodesRows>(p, s) : launch_fwd<false, kCodesRows>(p, s);
    default: return p.f32 ? launch_fwd<true, kCodesNone>(p, s) : launch_fwd<false, kCodesNone>(p, s);
    }
}

// As many workgroups as the card holds at once: each writes two rows of sums.
int block_norm_parts(int64_t rows, int64_t cols)
{
    const int waves = bwd_waves(cols), most = waves > 1 ? 4096 / waves : 1024;
    return (int)(rows < 1 ? 1 : rows < most ? rows : most);
}

hipError_t launch_block_norm_bwd(const BlockNormBwdParams &p, hipStream_t s)
{
    return p.f32 ? launch_bwd<true>(p, s) : launch_bwd<false>(p, s);
}

hipError_t launch_combine(const CombineParams &p, hipStream_t s)
{
    const int64_t total = p.T * (p.H / 8), want = (total + kThreads - 1) / kThreads;
    const dim3 g((unsigned)(want > (1 << 22) ? (1 << 22) : want)), b(kThreads);
    if (p.T * p.H * 2 * (p.k + 1) > kBlockStreamBytes) hipLaunchKernelGGL(combine_kernel<true>, g, b, 0, s, p);
    else hipLaunchKernelGGL(combine_kernel<false>, g, b, 0, s, p);
    return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineBwdParams &p, hipStream_t s)
{
    if (p.T * p.H * 2 * (2 * p.k + 1) > kBlockStreamBytes) return launch_combine_bwd_as<true>(p, s);
    return launch_combine_bwd_as<false>(p, s);
}

}  // namespace ptgg
