// few_tokens.hip -- the whole MoE layer for at most 64 tokens: router, FC1 +
// SwiGLU, FC2 and the weighted sum over each token's experts.
//
// The weights of the chosen experts are read once and everything else is
// small, so streaming them is the bound.  A wave owns 16 rows of one
// expert's matrix and reads each load instruction's 64 bytes of every row;
// the rows are the A operand of v_mfma_f32_16x16x32_bf16 (weights in 8 or 4
// bits are widened in registers, exactly), the expert's tokens the B operand,
// from LDS.  The order of the reduction is free, so a lane takes whichever
// consecutive elements its 16 bytes hold and reads the same ones of x.
//
// h = silu(gate) up is rounded to bf16 between the two products, as the grouped
// GEMM's SwiGLU epilogue does, so decoding and training see the same values.
#include "route_device.hpp"

namespace ptgg {

namespace {

constexpr int kFewLds = 65536;
constexpr int kRows = 16;                 // weight rows of a wave's tile
constexpr int kDepth = 4;                 // load instructions per buffer, two buffers

template <int WT>
struct Weights {
    static constexpr int lane_elems = WT == kFewBf16 ? 8 : WT == kFewMxfp8 ? 16 : 32;
    static constexpr int unit = 4 * lane_elems;           // elements of a row per load instruction
};

__host__ __device__ constexpr int lane_elems_of(int wt) { return wt == kFewBf16 ? 8 : wt == kFewMxfp8 ? 16 : 32; }
// LDS bytes of one token's row of K values: padded with zeros to whole units,
// and 16 bytes so that 16 rows start in different banks.
__host__ __device__ constexpr int x_pitch(int K, int wt)
{
    return (K + 4 * lane_elems_of(wt) - 1) / (4 * lane_elems_of(wt)) * (4 * lane_elems_of(wt)) * 2 + 16;
}
int row_cap(int K, int wt, int T)
{
    const int fit = kFewLds / x_pitch(K, wt);
    return fit < 16 ? (fit < T ? fit : T) : (T < 16 ? T : 16);
}

// What a lane loads of one unit.
template <int WT>
struct Unit {
    uintx4 w;
    uint32_t e;
};

template <int WT>
__device__ __forceinline__ Unit<WT> load_unit(const uint8_t *w, const uint8_t *s, int u, int g)
{
    Unit<WT> r;
    r.w = __builtin_nontemporal_load((const uintx4 *)(w + u * 64));
    r.e = 0;
    // blocks of 32: half of the unit (8 bits) or each lane's own (4 bits)
    if (WT == kFewMxfp8) r.e = s[2 * u + (g >> 1)];
    if (WT == kFewMxfp4) r.e = s[4 * u + g];
    return r;
}

// E8M0 byte to the power of two; 255 is NaN.
__device__ __forceinline__ float e8m0(uint32_t e)
{
    return e == 255u ? bits_f32(0x7FC00000u) : __builtin_ldexpf(1.0f, (int)e - 127);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

template <int WT>
__device__ __forceinline__ void mma_unit(const Unit<WT> &r, const uint8_t *x, floatx4 &acc0, floatx4 &acc1)
{
    // x: this lane's token and element group of the unit
    if constexpr (WT == kFewBf16) {
        acc0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, r.w), *(const bf16x8 *)x, acc0, 0,
                                                       0, 0);
    } else {
        const float f = e8m0(r.e);
        constexpr int N = WT == kFewMxfp8 ? 2 : 4;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            bf16x8 a;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf16x2_t v;
                if constexpr (WT == kFewMxfp8)
                    v = j & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[2 * i + (j >> 1)], f, true)
                              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[2 * i + (j >> 1)], f, false);
                else
                    v = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[i], f, 0)
                        : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[i], f, 1)
                        : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[i], f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[i], f, 3);
                a[2 * j] = v[0], a[2 * j + 1] = v[1];
            }
            floatx4 &acc = i & 1 ? acc1 : acc0;
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, *(const bf16x8 *)(x + 16 * i), acc, 0, 0, 0);
        }
    }
}

// Products of 16 weight rows with up to 16 tokens over K.  w, s: the row of
// lane % 16, from byte 16 (lane / 16) and from its scales; x: LDS row of token
// lane % 16, from the same elements.  Returns rows 4 (lane / 16) + 0..3 of
// token lane % 16.
template <int WT>
__device__ __forceinline__ floatx4 tile_product(const uint8_t *w, const uint8_t *s, const uint8_t *x, int K, int g)
{
    constexpr int UNIT = Weights<WT>::unit, XB = UNIT * 2;
    const int full = K / UNIT, tail = K % UNIT;
    floatx4 acc0 = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
    Unit<WT> a[kDepth], b[kDepth];
    if (full > 0) {
        const int last = full - 1;
#pragma unroll
        for (int i = 0; i < kDepth; ++i) a[i] = load_unit<WT>(w, s, min(i, last), g);
        for (int u = 0; u < full; u += 2 * kDepth) {
#pragma unroll
            for (int i = 0; i < kDepth; ++i) b[i] = load_unit<WT>(w, s, min(u + kDepth + i, last), g);
#pragma unroll
            for (int i = 0; i < kDepth; ++i)
                if (u + i < full) mma_unit<WT>(a[i], x + (u + i) * XB, acc0, acc1);
#pragma unroll
            for (int i = 0; i < kDepth; ++i) a[i] = load_unit<WT>(w, s, min(u + 2 * kDepth + i, last), g);
#pragma unroll
            for (int i = 0; i < kDepth; ++i)
                if (u + kDepth + i < full) mma_unit<WT>(b[i], x + (u + kDepth + i) * XB, acc0, acc1);
        }
    }
    if (tail) {
        // lanes past the row's end take zeros (x is zero there too)
        Unit<WT> r;
        r.w = uintx4{0, 0, 0, 0};
        r.e = 127;
        if (g * Weights<WT>::lane_elems < tail) r = load_unit<WT>(w, s, full, g);
        mma_unit<WT>(r, x + full * XB, acc0, acc1);
    }
    return acc0 + acc1;
}

// The rows of a block's tokens into LDS, zeros to the end of the last unit.
template <int NT, class Row>
__device__ __forceinline__ void stage_rows(uint8_t *lds, int pitch, int m, int K, Row row)
{
    const int pieces = (pitch - 16) / 16;
    for (int i = threadIdx.x; i < m * pieces; i += NT) {
        const int r = i / pieces, c = i % pieces;
        uintx4 v = {0, 0, 0, 0};
        if (c * 8 < K) v = *(const uintx4 *)(row(r) + c * 8);
        *(uintx4 *)(lds + r * pitch + c * 16) = v;
    }
}

// FC1 and SwiGLU: a tile is 8 gate rows and the 8 up rows of the same inner
// values, ordered so that a lane gets two gates and their two ups.
template <int WT>
__global__ __launch_bounds__(kThreads) void few_fc1_kernel(FewParams p)
{
    extern __shared__ __align__(16) uint8_t lds[];
    if ((int)blockIdx.y >= p.plan[0]) return;
    const intx4 blk = *(const intx4 *)(p.plan + 4 + 4 * blockIdx.y);
    const int e = blk[0], row0 = blk[1], m = blk[2], K = p.H;
    const int pitch = x_pitch(K, WT);
    stage_rows<kThreads>(lds, pitch, m, K,
                         [&](int r) { return p.x + (int64_t)p.route.token_of[row0 + r] * K; });
    __syncthreads();
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int j0 = ((int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6)) * 8;
    if (j0 >= p.I) return;
    const int row = ((r & 2) ? p.I : 0) + j0 + (r >> 2) * 2 + (r & 1);
    const int64_t at = (int64_t)e * 2 * p.I + row;
    const int64_t bytes = WT == kFewBf16 ? K * 2 : WT == kFewMxfp8 ? K : K / 2;
    const floatx4 c = tile_product<WT>(p.w1 + at * bytes + g * 16, p.w1s + at * (K / 32),
                                       lds + min(r, m - 1) * pitch + g * Weights<WT>::lane_elems * 2, K, g);
    if (r < m) {
        *(bf16x2_t *)(p.h + (int64_t)(row0 + r) * p.I + j0 + 2 * g) =
            bf16x2_t{(__bf16)silu_mul(c[0], c[2], p.swiglu_limit), (__bf16)silu_mul(c[1], c[3], p.swiglu_limit)};
    }
}

template <int WT>
__global__ __launch_bounds__(kThreads) void few_fc2_kernel(FewParams p)
{
    extern __shared__ __align__(16) uint8_t lds[];
    if ((int)blockIdx.y >= p.plan[0]) return;
    const intx4 blk = *(const intx4 *)(p.plan + 4 + 4 * blockIdx.y);
    const int e = blk[0], row0 = blk[1], m = blk[2], K = p.I;
    const int pitch = x_pitch(K, WT);
    stage_rows<kThreads>(lds, pitch, m, K, [&](int r) { return p.h + (int64_t)(row0 + r) * K; });
    __syncthreads();
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int n0 = ((int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6)) * kRows;
    if (n0 >= p.H) return;
    const int64_t at = (int64_t)e * p.H + min(n0 + r, p.H - 1);
    const int64_t bytes = WT == kFewBf16 ? K * 2 : WT == kFewMxfp8 ? K : K / 2;
    const floatx4 c = tile_product<WT>(p.w2 + at * bytes + g * 16, p.w2s + at * (K / 32),
                                       lds + min(r, m - 1) * pitch + g * Weights<WT>::lane_elems * 2, K, g);
    if (r < m && n0 + 4 * g < p.H) *(floatx4 *)(p.y + (int64_t)(row0 + r) * p.H + n0 + 4 * g) = c;
}

// out[t] = sum over the slots, in their order, of weight times the expert's row.
__global__ __launch_bounds__(kThreads) void few_sum_kernel(FewParams p)
{
    const int t = blockIdx.y, c = ((int)blockIdx.x * kThreads + (int)threadIdx.x) * 4;
    if (c >= p.H) return;
    floatx4 sum = {0, 0, 0, 0};
    for (int j = 0; j < p.k; ++j) {
        const int row = p.route.row_of[t * p.k + j];
        if (row < 0) continue;
        const float w = p.route.topk_weights[t * p.k + j];
        const floatx4 v = *(const floatx4 *)(p.y + (int64_t)row * p.H + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(w, v[i], sum[i]);
    }
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *(bf16x4 *)((__bf16 *)p.out + (int64_t)t * p.H + c) =
        bf16x4{(__bf16)sum[0], (__bf16)sum[1], (__bf16)sum[2], (__bf16)sum[3]};
}

template <int WT>
hipError_t launch_products(const FewParams &p, int cap, hipStream_t s)
{
    // the grid covers the most blocks the routing can give; the rest leave at once
    const int pairs = p.T * p.k, split = p.E < pairs ? p.E : pairs;
    int blocks = split + pairs / cap;
    if (blocks > pairs) blocks = pairs;
    constexpr int W = kThreads / 64;
    const unsigned t1 = (unsigned)((p.I / 8 + W - 1) / W), t2 = (unsigned)(((p.H + kRows - 1) / kRows + W - 1) / W);
    hipLaunchKernelGGL(few_fc1_kernel<WT>, dim3(t1, (unsigned)blocks), dim3(kThreads), cap * x_pitch(p.H, WT), s, p);
    hipLaunchKernelGGL(few_fc2_kernel<WT>, dim3(t2, (unsigned)blocks), dim3(kThreads), cap * x_pitch(p.I, WT), s, p);
    hipLaunchKernelGGL(few_sum_kernel, dim3((unsigned)((p.H / 4 + kThreads - 1) / kThreads), (unsigned)p.T),
                       dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace

int few_max_blocks(int T, int E, int k) { return T * k; }

hipError_t launch_few_tokens(const FewParams &p, hipStream_t s)
{
    const int c1 = row_cap(p.H, p.weights, p.T), c2 = row_cap(p.I, p.weights, p.T);
    const int cap = c1 < c2 ? c1 : c2;
    hipError_t e = launch_moe_route_plan(p.route, RoutePlan{p.plan, cap}, s);
    if (e != hipSuccess) return e;
    switch (p.weights) {
    case kFewMxfp8: return launch_products<kFewMxfp8>(p, cap, s);
    case kFewMxfp4: return launch_products<kFewMxfp4>(p, cap, s);
    default: return launch_products<kFewBf16>(p, cap, s);
    }
}

}  // namespace ptgg
