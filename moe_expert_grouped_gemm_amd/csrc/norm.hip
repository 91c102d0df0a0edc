// norm.hip -- RMS norm of the residual stream, forward and backward.
//
// Forward, per row: h = x + residual, rounded once to the stream's type and
// written back as the stream; rstd = (mean(h^2) + eps)^-1/2; v = h rstd w in
// fp32.  v leaves rounded to bf16 (y) and, from the same unrounded fp32 value,
// as E4M3 codes: blocks of 32 with an E8M0 exponent, or one fp32 factor per
// row, by the rules of the stand-alone quantisers.  Codes taken from v rather
// than from y round once instead of twice.
//
// Backward, per row, with c = rstd^2 / cols * sum(dy w h):
//     ds = dres + rstd (dy w - h c),      dw = sum over rows of dy h rstd.
//
// Both read and write each element once: the whole row stays in registers
// between its sum and its outputs, so memory traffic is the bound.
#include "common.hpp"
#include "layer.hpp"

namespace ptgg {

namespace {

// Traffic from which a call's rows go past the caches.
constexpr int64_t kNormStreamBytes = (int64_t)80 << 20;

// Sum over the wave, in every lane: four DPP steps inside each 16 lanes, then
// the four rows' sums by readlane.
__device__ __forceinline__ float wave_sum(float x)
{
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0xB1, 0xF, 0xF, false));    // lanes ^ 1
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0x4E, 0xF, 0xF, false));    // lanes ^ 2
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0x141, 0xF, 0xF, false));   // mirror of 8
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0x140, 0xF, 0xF, false));   // mirror of 16
    const int i = (int)f32_bits(x);
    return (bits_f32(__builtin_amdgcn_readlane(i, 0)) + bits_f32(__builtin_amdgcn_readlane(i, 16))) +
           (bits_f32(__builtin_amdgcn_readlane(i, 32)) + bits_f32(__builtin_amdgcn_readlane(i, 48)));
}

__device__ __forceinline__ uint32_t quad_max_u32(uint32_t x)
{
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x)
{
    x = quad_max_u32(x);
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, false));
    return max(max((uint32_t)__builtin_amdgcn_readlane((int)x, 0), (uint32_t)__builtin_amdgcn_readlane((int)x, 16)),
               max((uint32_t)__builtin_amdgcn_readlane((int)x, 32), (uint32_t)__builtin_amdgcn_readlane((int)x, 48)));
}

// Across the W waves of a row's team (the whole workgroup where W > 1), in a
// fixed order; s holds W words that no other reduction in flight uses.
template <int W>
__device__ __forceinline__ float team_sum(float x, float *s)
{
    x = wave_sum(x);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        x = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w) x += s[w];
    }
    return x;
}

template <int W>
__device__ __forceinline__ uint32_t team_max_u32(uint32_t x, uint32_t *s)
{
    x = wave_max_u32(x);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        x = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w) x = max(x, s[w]);
    }
    return x;
}

__device__ __forceinline__ void unpack8(const uintx4 v, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bits_f32(v[i] << 16);
        f[2 * i + 1] = bits_f32(v[i] & 0xFFFF0000u);
    }
}

// bf16 to nearest even; a NaN stays a (quiet) NaN.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

__device__ __forceinline__ uintx4 pack8(const float (&f)[8])
{
    return uintx4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
}

// E4M3 within +-448; NaN stays NaN.
__device__ __forceinline__ float clamp448(float v)
{
    const float c = __builtin_fminf(__builtin_fmaxf(v, -448.0f), 448.0f);
    return v != v ? v : c;
}

__device__ __forceinline__ uintx2 codes8(const float (&f)[8])
{
    int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[0]), clamp448(f[1]), 0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[2]), clamp448(f[3]), w0, true);
    int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[4]), clamp448(f[5]), 0, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[6]), clamp448(f[7]), w1, true);
    return uintx2{(uint32_t)w0, (uint32_t)w1};
}

__device__ __forceinline__ uint32_t amax8(const float (&f)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, f32_bits(f[i]) & 0x7FFFFFFFu);
    return m;
}

// Loads and stores, past the caches with NT -- where a lane's 16 bytes are all
// that it reads there: of 8 fp32 values two instructions read half a line each,
// and the second must find it in the caches.
template <bool NT, class T>
__device__ __forceinline__ T load_as(const void *p)
{
    return NT ? __builtin_nontemporal_load((const T *)p) : *(const T *)p;
}
template <bool NT, class T>
__device__ __forceinline__ void store_as(void *p, T v)
{
    if (NT) __builtin_nontemporal_store(v, (T *)p);
    else *(T *)p = v;
}

// Eight values of the residual stream from element e.
template <bool F32, bool NT>
__device__ __forceinline__ void load_stream(const void *p, int64_t e, float (&f)[8])
{
    if constexpr (F32) {
        const floatx4 a = *(const floatx4 *)((const float *)p + e), b = *(const floatx4 *)((const float *)p + e + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
    } else {
        unpack8(load_as<NT, uintx4>((const uint16_t *)p + e), f);
    }
}

template <bool F32, bool NT>
__device__ __forceinline__ void store_stream(void *p, int64_t e, const float (&f)[8])
{
    if constexpr (F32) {
        *(floatx4 *)((float *)p + e) = floatx4{f[0], f[1], f[2], f[3]};
        *(floatx4 *)((float *)p + e + 4) = floatx4{f[4], f[5], f[6], f[7]};
    } else {
        store_as<NT>((uint16_t *)p + e, pack8(f));
    }
}

// W waves hold one row, NV groups of 8 values per lane (group i of lane t is
// group i * 64 W + t of the row, so a block of 32 is one quad of lanes).
template <bool F32, int CODES, int W, int NV, bool NT>
__global__ __launch_bounds__(kThreads) void rmsnorm_fwd_kernel(NormFwdParams p)
{
    constexpr int TEAM = 64 * W, ROWS = kThreads / TEAM;
    __shared__ float s_sum[4];
    __shared__ uint32_t s_max[4];
    const int t = (int)threadIdx.x % TEAM;
    const int64_t r = (int64_t)blockIdx.x * ROWS + (int)threadIdx.x / TEAM;
    if (r >= p.rows) return;                 // whole teams: W > 1 has one row per workgroup
    const int n8 = p.cols >> 3;
    const int64_t base = r * p.cols;
    float h[NV][8];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = i * TEAM + t;
        if (g < n8) {
            unpack8(load_as<NT, uintx4>(p.x + base + g * 8), h[i]);
            if (p.residual) {
                float d[8];
                load_stream<F32, NT>(p.residual, base + g * 8, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] += d[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
        }
        // the sum is rounded to the stream's type before it is used: the norm
        // is of the stream that the next layer reads
        if constexpr (!F32) {
            const uintx4 b = pack8(h[i]);
            if (p.residual_out && g < n8) store_as<NT>((uint16_t *)p.residual_out + base + g * 8, b);
            unpack8(b, h[i]);
        } else {
            if (p.residual_out && g < n8) store_stream<true, NT>(p.residual_out, base + g * 8, h[i]);
        }
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) part = __builtin_fmaf(h[i][j], h[i][j], part);
        sq += part;
    }
    sq = team_sum<W>(sq, s_sum);
    const float rstd = 1.0f / __builtin_sqrtf(sq / (float)p.cols + p.eps);
    if (t == 0 && p.rstd) p.rstd[r] = rstd;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = i * TEAM + t;
        if (g < n8) {
            float w[8];
            unpack8(*(const uintx4 *)(p.weight + g * 8), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * rstd * w[j];
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
        // fminf would turn a NaN factor into a number
        const float scale = mf != mf ? mf : f;
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
void launch_fwd_as(const NormFwdParams &p, hipStream_t s)
{
    const int n8 = p.cols / 8;
    const dim3 b(kThreads);
#define PTGG_NORM(W, NV)                                                                                        \
    hipLaunchKernelGGL((rmsnorm_fwd_kernel<F32, CODES, W, NV, NT>),                                             \
                       dim3((unsigned)((p.rows + 4 / W - 1) / (4 / W))), b, 0, s, p)
    // a wave per row leaves a workgroup's lanes idle least where rows are short (16000 x 288 fp32: 12.6 us against
    // 16.5 for a workgroup per row; 1021 x 2880: 10.9 against 8.8)
    if (n8 <= 64) PTGG_NORM(1, 1);
    else if (n8 <= 128) PTGG_NORM(1, 2);
    else if (n8 <= 256) PTGG_NORM(4, 1);
    else if (n8 <= 512) PTGG_NORM(4, 2);
    else if (n8 <= 768) PTGG_NORM(4, 3);
    else if (n8 <= 1024) PTGG_NORM(4, 4);
    else if (n8 <= 2048) PTGG_NORM(4, 8);
    else PTGG_NORM(4, 16);
#undef PTGG_NORM
}

template <bool F32, int CODES>
hipError_t launch_fwd(const NormFwdParams &p, hipStream_t s)
{
    // what the caches cannot hold anyway goes past them, but for the codes, which the next product reads (bf16 stream:
    // 8192 x 4096 with MXFP8 codes, 302 MB: 50.6 us against 59.7; 3000 x 4064, 98 MB: 22.3 against 24.3; 5000 x 1056,
    // 47 MB: 13.5 against 11.6)
    const int64_t bytes = p.rows * p.cols * (F32 ? 12 : 8);
    if (bytes > kNormStreamBytes) launch_fwd_as<F32, CODES, true>(p, s);
    else launch_fwd_as<F32, CODES, false>(p, s);
    return hipGetLastError();
}

// The loads of a row's share as they come, so that the next row's can be in
// flight while this one is worked on.
template <bool F32, int TEAM, int NV, bool NT>
struct RowLoads {
    static constexpr int SV = F32 ? 2 : 1;               // 16-byte loads per 8 stream values
    uintx4 dy[NV], s[NV * SV], dres[NV * SV];
    float rstd;
    __device__ __forceinline__ void load(const NormBwdParams &p, int64_t r, int t)
    {
        const int64_t base = r * p.cols;
        rstd = p.rstd[r];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TEAM + t) * 8;
            if (e < p.cols) {
                dy[i] = load_as<NT, uintx4>(p.dy + base + e);
                const int64_t at = (base + e) * (F32 ? 4 : 2);
#pragma unroll
                for (int j = 0; j < SV; ++j) {
                    s[i * SV + j] = load_as<NT && !F32, uintx4>((const uint8_t *)p.s + at + 16 * j);
                    if (p.dres) dres[i * SV + j] = load_as<NT && !F32, uintx4>((const uint8_t *)p.dres + at + 16 * j);
                }
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

// Backward: W waves hold a row (8 where it is long); a workgroup's teams
// take rows a grid apart and keep their lanes' weight gradients in registers.
// Its teams' are added in order, and with more than one part the parts' go to
// the workspace, where rmsnorm_dweight_kernel adds them in order.
__host__ __device__ constexpr int bwd_threads(int W) { return W > 4 ? 64 * W : kThreads; }
template <bool F32, int W, int NV, bool NT>
__global__ __launch_bounds__(bwd_threads(W)) void rmsnorm_bwd_kernel(NormBwdParams p, int parts)
{
    constexpr int TEAM = 64 * W, TEAMS = bwd_threads(W) / TEAM;
    __shared__ float s_sum[2][W];
    __shared__ floatx4 s_dw[TEAMS > 1 ? (TEAMS - 1) * TEAM * NV * 2 : 1];
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    float dw[NV][8] = {};
    int flip = 0;
    const int64_t first = (int64_t)blockIdx.x * TEAMS + team, step = (int64_t)parts * TEAMS;
    constexpr bool AHEAD = W <= 4;                       // long rows fill the registers
    RowLoads<F32, TEAM, NV, NT> next;
    if (AHEAD && first < p.rows) next.load(p, first, t);
    for (int64_t r = first; r < p.rows; r += step, flip ^= 1) {
        const int64_t base = r * p.cols;
        RowLoads<F32, TEAM, NV, NT> row;
        if constexpr (AHEAD) {
            row = next;
            if (r + step < p.rows) next.load(p, r + step, t);
        } else {
            row.load(p, r, t);
        }
        float h[NV][8], g[NV][8];
        const float rstd = row.rstd;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TEAM + t) * 8;
            if (e < p.cols) {
                float w[8];
                unpack8(row.dy[i], g[i]);
                row.widen(row.s + i * row.SV, h[i]);
                unpack8(*(const uintx4 *)(p.weight + e), w);
                float part = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[i][j] = __builtin_fmaf(g[i][j], h[i][j] * rstd, dw[i][j]);
                    g[i][j] *= w[j];
                    part = __builtin_fmaf(g[i][j], h[i][j], part);
                }
                dot += part;
            }
        }
        // two sets of words: the next row's sums never meet readers of this one's
        dot = team_sum<W>(dot, s_sum[flip]);
        const float c = rstd * rstd * (dot / (float)p.cols);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TEAM + t) * 8;
            if (e < p.cols) {
                float d[8] = {};
                if (p.dres) row.widen(row.dres + i * row.SV, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] += rstd * (g[i][j] - h[i][j] * c);
                store_stream<F32, NT>(p.ds, base + e, d);
            }
        }
    }
    if (!p.dweight) return;
    if constexpr (TEAMS > 1) {
        if (team) {
            floatx4 *out = s_dw + (team - 1) * TEAM * NV * 2 + t;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                out[(2 * i) * TEAM] = floatx4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
                out[(2 * i + 1) * TEAM] = floatx4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
            }
        }
        __syncthreads();
        if (team) return;
#pragma unroll
        for (int k = 1; k < TEAMS; ++k) {
            const floatx4 *in = s_dw + (k - 1) * TEAM * NV * 2 + t;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) dw[i][j] += in[(2 * i + j / 4) * TEAM][j & 3];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TEAM + t) * 8;
        if (e >= p.cols) continue;
        float *out = parts > 1 ? p.partials + (int64_t)blockIdx.x * p.cols + e : p.dweight + e;
        if (parts == 1 && p.accumulate) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[i][j] += out[j];
        }
        store_stream<true, false>(out, 0, dw[i]);
    }
}

// dweight[c] (+)= the parts' sums.  A workgroup takes 32 columns: 8 lanes of
// four, 128 rows of parts side by side, joined in LDS in their order.
constexpr int kJoinThreads = 1024, kJoinCols = 32;
__global__ __launch_bounds__(kJoinThreads) void rmsnorm_dweight_kernel(const float *__restrict__ partials,
                                                                       float *dweight, int parts, int cols,
                                                                       int accumulate)
{
    constexpr int SIDE = kJoinThreads / (kJoinCols / 4);
    __shared__ floatx4 s[SIDE][kJoinCols / 4 + 1];
    const int lane = threadIdx.x % (kJoinCols / 4), side = threadIdx.x / (kJoinCols / 4);
    const int c = (int)blockIdx.x * kJoinCols + lane * 4;
    floatx4 sum = {0, 0, 0, 0};
    if (c < cols) {
#pragma unroll 4
        for (int i = side; i < parts; i += SIDE) sum += *(const floatx4 *)(partials + (int64_t)i * cols + c);
    }
    s[side][lane] = sum;
    __syncthreads();
    for (int n = SIDE / 2; n >= 1; n /= 2) {
        if (side < n) s[side][lane] += s[side + n][lane];
        __syncthreads();
    }
    if (side == 0 && c < cols) {
        floatx4 *out = (floatx4 *)(dweight + c);
        *out = accumulate ? *out + s[0][lane] : s[0][lane];
    }
}

template <bool F32, bool NT>
hipError_t launch_bwd_as(const NormBwdParams &p, hipStream_t s)
{
    const int n8 = p.cols / 8, parts = norm_bwd_parts(p.rows);
#define PTGG_NORM(W, NV)                                                                                        \
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<F32, W, NV, NT>), dim3((unsigned)parts), dim3(bwd_threads(W)), 0, s, p, \
                       parts)
    if (n8 <= 64) PTGG_NORM(1, 1);
    else if (n8 <= 128) PTGG_NORM(1, 2);
    else if (n8 <= 256) PTGG_NORM(4, 1);
    else if (n8 <= 512) PTGG_NORM(4, 2);
    else if (n8 <= 768) PTGG_NORM(4, 3);
    else if (n8 <= 1024) PTGG_NORM(4, 4);
    else if (n8 <= 2048) PTGG_NORM(8, 4);
    else PTGG_NORM(8, 8);
#undef PTGG_NORM
    if (parts > 1 && p.dweight)
        hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((unsigned)((p.cols + kJoinCols - 1) / kJoinCols)),
                           dim3(kJoinThreads), 0, s, p.partials, p.dweight, parts, p.cols, p.accumulate);
    return hipGetLastError();
}

template <bool F32>
hipError_t launch_bwd(const NormBwdParams &p, hipStream_t s)
{
    const int64_t bytes = p.rows * p.cols * (F32 ? 14 : 8);
    return bytes > kNormStreamBytes ? launch_bwd_as<F32, true>(p, s) : launch_bwd_as<F32, false>(p, s);
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const NormFwdParams &p, hipStream_t s)
{
    switch (p.codes) {
    case kCodesMx: return p.f32 ? launch_fwd<true, kCodesMx>(p, s) : launch_fwd<false, kCodesMx>(p, s);
    case kCodesRows: return p.f32 ? launch_fwd<true, kCodesRows>(p, s) : launch_fwd<false, kCodesRows>(p, s);
    default: return p.f32 ? launch_fwd<true, kCodesNone>(p, s) : launch_fwd<false, kCodesNone>(p, s);
    }
}

int norm_bwd_parts(int64_t rows)
{
    // a few rows one workgroup adds up itself, which saves a launch (4 x 4064 fp32: 6.7 us against 8.8, 8: 11.6 against
    // 8.9)
    if (rows <= 5) return 1;
    // each part's row of sums is written and read again, too few parts leave the card idle (517 x 4096 fp32: 13.0 us
    // with 256, 14.0 with 512; 4000 x 2016: 30.0 and 26.6; 16384 x 2880: 81 with 512, 76 with 1024)
    const int64_t most = rows < 1024 ? 256 : rows < 4096 ? 512 : 1024;
    return (int)(rows < most ? rows : most);
}

hipError_t launch_rmsnorm_bwd(const NormBwdParams &p, hipStream_t s)
{
    return p.f32 ? launch_bwd<true>(p, s) : launch_bwd<false>(p, s);
}

}  // namespace ptgg
