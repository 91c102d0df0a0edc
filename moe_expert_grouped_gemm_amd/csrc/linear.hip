// linear.hip -- dense matrix product with bias, activation and residual in its
// epilogue, its data gradient (which ends in the activation's gradient) and its
// weight gradient.
//
//   forward  C[m, n] = sum_k x[m, k] w[n, k]      both operands along the reduction
//   dgrad    C[m, k] = sum_n dy[m, n] w[n, k]     w across it
//   wgrad    C[n, k] = sum_m dy[m, n] x[m, k]     both across it
//
// A workgroup computes a TM x TN tile of C over one part of the reduction, in
// stages of 64 values through a ring of LDS slots filled by direct loads.
// Operands keep in LDS the layout that they have in memory: along the reduction
// as rows of 128 bytes, across it as 64 rows of the tile's columns, which lanes
// read transposed (ds_read_b64_tr_b16) or, in the widest tile, turn themselves.
// Products are bf16 matrix instructions with the operands swapped, so that a
// lane holds four neighbouring columns of one row and the tile passes through
// LDS in 16-byte pieces, still in fp32: bias, activation and residual are
// applied to unrounded sums and the result is rounded once.  Where the tiles
// alone do not fill the chip the reduction is cut in parts whose fp32 sums a
// second kernel adds in order and finishes.
//
// What bounds them: products that fill the chip the matrix cores at the clock
// that the power limit leaves them (8192^3: 1506 TFLOP/s at 1.5 to 1.8 GHz, 2.4
// when idle); those of some hundred rows the loads into LDS, about 84 GB/s to a
// CU while its stages run, which is near the most that direct loads bring in, and
// the waits of a start and an end (1021 x 2880 x 2880: 24 us, 7 of them start and
// end); those of few rows memory (1 x 4096 x 4096: 3.5 TB/s, launch included).
#include <utility>

#include "dense.hpp"
#include "linear_plan.hpp"
#include "pipeline.hpp"
#include "rows.hpp"

namespace ptgg {

namespace {

template <int V>
struct IC { static constexpr int value = V; };

template <class F, int... I>
__device__ __forceinline__ void unrolled(F &&f, std::integer_sequence<int, I...>)
{
    (f(IC<I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(F &&f)
{
    unrolled((F &&)f, std::make_integer_sequence<int, N>{});
}

constexpr int kWideRows = kWide;              // most rows of a tile

// ------------------------------------------------------------------ activations
// e^x by the hardware's 2^x.  The rounding of x log2(e) makes it |x| 2^-24 off,
// relative: in what it is used for, sigmoids of c times c, less than an ulp of
// |c| + 1.  Past the type's range it is 0 or infinite, of a NaN a NaN.
__device__ __forceinline__ float exp_(float x) { return __builtin_amdgcn_exp2f(1.44269502162933349609375f * x); }
__device__ __forceinline__ float sigmoid_(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_(-x)); }

constexpr float kSqrtHalf = 0.707106769084930419921875f;
constexpr float kTwoBeta = 1.59576916694641113281f;        // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

__device__ __forceinline__ float act_of(float c, int act)
{
    switch (act) {
    case kActSilu: return c * sigmoid_(c);
    case kActGelu: return 0.5f * c * erfcf(-kSqrtHalf * c);
    // (1 + tanh u) / 2 = sigmoid(2 u)
    case kActGeluTanh: return c * sigmoid_(kTwoBeta * (c + kCube * c * c * c));
    case kActRelu2: return c > 0.0f ? c * c : c != c ? c : 0.0f;
    default: return c;
    }
}

__device__ __forceinline__ float act_slope(float c, int act)
{
    float d = 1.0f;
    switch (act) {
    case kActSilu: {
        const float s = sigmoid_(c);
        d = s * (1.0f + c * (1.0f - s));
        break;
    }
    case kActGelu: d = 0.5f * erfcf(-kSqrtHalf * c) + c * (0.3989422804f * exp_(-0.5f * c * c)); break;
    case kActGeluTanh: {
        const float s = sigmoid_(kTwoBeta * (c + kCube * c * c * c));
        // far out s (1 - s) is 0 where its factor may be infinite
        const float t = s * (1.0f - s);
        d = t == 0.0f ? s : s + c * t * (kTwoBeta * (1.0f + 3.0f * kCube * c * c));
        break;
    }
    case kActRelu2: d = c > 0.0f ? 2.0f * c : 0.0f; break;
    default: return 1.0f;
    }
    return c != c ? c : d;
}

// SwiGLU's clamp: a gate at most lim, an up within [-lim, lim]; NaN stays.
__device__ __forceinline__ void glu8(float (&g)[8], float (&u)[8], float lim)
{
    if (lim < __builtin_huge_valf()) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = g[i] > lim ? lim : g[i];
            u[i] = u[i] > lim ? lim : u[i] < -lim ? -lim : u[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = g[i] * sigmoid_(g[i]) * u[i];
}
// g, u: the saved gates and ups, then their gradients for d, those of the products
__device__ __forceinline__ void glu_slope8(float (&g)[8], float (&u)[8], const float (&d)[8], float lim)
{
    uint32_t shut = 0;                   // bits of gates and ups that the clamp holds: no gradient into them
    if (lim < __builtin_huge_valf()) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            shut |= (g[i] > lim ? 1u : 0u) << i | (__builtin_fabsf(u[i]) > lim ? 1u : 0u) << (8 + i);
            g[i] = g[i] > lim ? lim : g[i];
            u[i] = u[i] > lim ? lim : u[i] < -lim ? -lim : u[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = sigmoid_(g[i]), dg = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
        u[i] = d[i] * (g[i] * s);
        g[i] = dg;
    }
    if (shut) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (shut >> i & 1) g[i] = 0.0f;
            if (shut >> (8 + i) & 1) u[i] = 0.0f;
        }
    }
}

__device__ __forceinline__ void act8(float (&v)[8], int act)
{
    switch (act) {                       // one branch for the eight
#define PTGG_ACT(A)                                                           \
    case A:                                                                   \
        _Pragma("unroll") for (int i = 0; i < 8; ++i) v[i] = act_of(v[i], A); \
        break;
        PTGG_ACT(kActSilu)
        PTGG_ACT(kActGelu)
        PTGG_ACT(kActGeluTanh)
        PTGG_ACT(kActRelu2)
#undef PTGG_ACT
    default: break;
    }
}

__device__ __forceinline__ void slope8(float (&v)[8], const float (&c)[8], int act)
{
    switch (act) {
#define PTGG_ACT(A)                                                               \
    case A:                                                                       \
        _Pragma("unroll") for (int i = 0; i < 8; ++i) v[i] *= act_slope(c[i], A); \
        break;
        PTGG_ACT(kActSilu)
        PTGG_ACT(kActGelu)
        PTGG_ACT(kActGeluTanh)
        PTGG_ACT(kActRelu2)
#undef PTGG_ACT
    default: break;
    }
}

// ------------------------------------------------------------------ finish
// What becomes of eight neighbouring sums of a row.  Sums are fp32 until the one
// rounding of each output.  v: the sums from some column of the product on, u,
// for kFinFwdGlu: those of the ups, N / 2 columns on; afterwards the outputs.
struct Extra {
    uintx4 r[2];                          // residual, as it lies in memory (bf16: r[0])
    uintx4 c[2];                          // kFinGrad*: the saved sums, of gates and ups
};
struct Saved {
    uintx4 v, u;                          // kFinFwd*: the sums with bias, in bf16
};

template <int FIN, bool F32>
__device__ __forceinline__ Saved finish8(const FinishParams &p, const float (&bias)[8], const float (&bias_u)[8], const Extra &x,
                                         float (&v)[8], float (&u)[8])
{
    Saved saved = {};
    if constexpr (FIN == kFinFwd || FIN == kFinFwdGlu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += bias[i];
        saved.v = pack8(v);
        if constexpr (FIN == kFinFwdGlu) {
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] += bias_u[i];
            saved.u = pack8(u);
            glu8(v, u, p.limit);
        } else {
            act8(v, p.act);
        }
    } else if constexpr (FIN == kFinGrad) {
        float c[8];
        unpack8(x.c[0], c);
        slope8(v, c, p.act);
    } else {
        float g[8], w[8];
        unpack8(x.c[0], g);
        unpack8(x.c[1], w);
        glu_slope8(g, w, v, p.limit);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = g[i], u[i] = w[i];
    }
    if constexpr (FIN != kFinGradGlu) {                    // zeros where there is none
        float f[8];
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = bits_f32(x.r[0][i]), f[4 + i] = bits_f32(x.r[1][i]);
        } else {
            unpack8(x.r[0], f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
    }
    return saved;
}

template <int FIN>
__device__ __forceinline__ void load_bias8(const FinishParams &p, int64_t n, float (&bias)[8], float (&bias_u)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = bias_u[i] = 0.0f;
    if ((FIN == kFinFwd || FIN == kFinFwdGlu) && p.bias) {
        unpack8(*(const uintx4 *)(p.bias + n), bias);
        if (FIN == kFinFwdGlu) unpack8(*(const uintx4 *)(p.bias + (p.N >> 1) + n), bias_u);
    }
}

// One row, from its sums to memory.
template <int FIN, bool F32>
__device__ __forceinline__ void finish_row_as(const FinishParams &p, int64_t m, int64_t n, float (&v)[8], float (&u)[8])
{
    const int64_t at = m * p.ldo + n;
    float bias[8], bias_u[8];
    load_bias8<FIN>(p, n, bias, bias_u);
    Extra x = {};
    if (FIN != kFinGradGlu && p.residual) {
        x.r[0] = *(const uintx4 *)((const uint8_t *)p.residual + at * (F32 ? 4 : 2));
        if (F32) x.r[1] = *(const uintx4 *)((const uint8_t *)p.residual + at * 4 + 16);
    }
    if ((FIN == kFinGrad && p.c) || FIN == kFinGradGlu) x.c[0] = *(const uintx4 *)(p.c + at);
    if (FIN == kFinGradGlu) x.c[1] = *(const uintx4 *)(p.c + at + p.N);
    const Saved s = finish8<FIN, F32>(p, bias, bias_u, x, v, u);
    if ((FIN == kFinFwd || FIN == kFinFwdGlu) && p.save) {
        *(uintx4 *)(p.save + m * p.N + n) = s.v;
        if (FIN == kFinFwdGlu) *(uintx4 *)(p.save + m * p.N + (p.N >> 1) + n) = s.u;
    }
    store_stream<F32, false>(p.out, at, v);
    if (FIN == kFinGradGlu) store_stream<false, false>(p.out, at + p.N, u);
}

template <int FIN>
__device__ __forceinline__ void finish_row(const FinishParams &p, int64_t m, int64_t n, float (&v)[8], float (&u)[8])
{
    if (FIN < kFinGrad && p.f32) finish_row_as<FIN, true>(p, m, n, v, u);
    else finish_row_as<FIN, false>(p, m, n, v, u);
}

// 16 bytes of a buffer at `base`; at or past `bytes` zeros are read and nothing is
// written.  Plain functions: see dma16.
__device__ __forceinline__ uintx4 buf_load(const void *base, uint32_t bytes, uint32_t voff, uint32_t soff)
{
    return __builtin_bit_cast(uintx4, __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(base, bytes), voff, soff, 0));
}
__device__ __forceinline__ void buf_store(uintx4 v, const void *base, uint32_t bytes, uint32_t voff, uint32_t soff)
{
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), make_rsrc(base, bytes), voff, soff, 0);
}

// Rows of a wave from row m0 on, each lane at its 8 columns.  Loads and stores
// have no branch around them -- what is not there has a bound of 0 -- so that the
// wait for a row's loads is a count that leaves the stores in flight (with a
// branch it was for every store before: 1000 cycles a row, 38000 cycles a tile of
// 256 x 256 with its copies unrolled, now 18600).
template <int FIN, bool F32>
struct FinishRows {
    static constexpr bool FWD = FIN == kFinFwd || FIN == kFinFwdGlu;
    const FinishParams &p;
    const uint8_t *out, *res, *sv, *cs;
    uint32_t out_b, res_b, sv_b, cs_b;    // bounds
    uint32_t vo, vs;                      // this lane's offsets in out (and residual and c) and in save
    uint32_t ldo_b, lds_b;                // bytes of a row
    uint32_t far_o, far_s;                // from the gates' columns to the ups'
    float bias[8], bias_u[8];

    __device__ __forceinline__ FinishRows(const FinishParams &f, int64_t m0, int64_t M, int r0, int64_t n, bool live) : p(f)
    {
        const int rows = (int)min(M - m0, (int64_t)kWideRows);
        constexpr uint32_t SIZE = F32 ? 4 : 2;
        ldo_b = (uint32_t)f.ldo * SIZE;
        lds_b = (uint32_t)f.N * 2;
        out = (const uint8_t *)f.out + m0 * ldo_b;
        out_b = rows > 0 ? rows * ldo_b : 0;
        res = (const uint8_t *)f.residual + m0 * ldo_b;
        res_b = f.residual ? out_b : 0;
        sv = (const uint8_t *)f.save + m0 * lds_b;
        sv_b = f.save && rows > 0 ? rows * lds_b : 0;
        cs = (const uint8_t *)f.c + m0 * ldo_b;
        cs_b = f.c ? out_b : 0;
        vo = live ? r0 * ldo_b + (uint32_t)n * SIZE : kOOB;
        vs = live ? r0 * lds_b + (uint32_t)n * 2 : kOOB;
        far_o = (uint32_t)f.N * 2;
        far_s = (uint32_t)f.N;            // N / 2 columns
        load_bias8<FIN>(f, live ? n : 0, bias, bias_u);
    }
    // `row` rows after this lane's first
    __device__ __forceinline__ void fetch(Extra &x, uint32_t row) const
    {
        const uint32_t s = row * ldo_b;
        if (FIN != kFinGradGlu) x.r[0] = buf_load(res, res_b, vo, s);
        if (F32) x.r[1] = buf_load(res, res_b, vo, s + 16);
        if (!FWD) x.c[0] = buf_load(cs, cs_b, vo, s);
        if (FIN == kFinGradGlu) x.c[1] = buf_load(cs, cs_b, vo, s + far_o);
    }
    __device__ __forceinline__ void store(const Extra &x, uint32_t row, float (&v)[8], float (&u)[8]) const
    {
        const Saved sv8 = finish8<FIN, F32>(p, bias, bias_u, x, v, u);
        const uint32_t s = row * ldo_b;
        if (FWD) buf_store(sv8.v, sv, sv_b, vs, row * lds_b);
        if (FIN == kFinFwdGlu) buf_store(sv8.u, sv, sv_b, vs, row * lds_b + far_s);
        if constexpr (F32) {
            buf_store(uintx4{f32_bits(v[0]), f32_bits(v[1]), f32_bits(v[2]), f32_bits(v[3])}, out, out_b, vo, s);
            buf_store(uintx4{f32_bits(v[4]), f32_bits(v[5]), f32_bits(v[6]), f32_bits(v[7])}, out, out_b, vo, s + 16);
        } else {
            buf_store(pack8(v), out, out_b, vo, s);
        }
        if (FIN == kFinGradGlu) buf_store(pack8(u), out, out_b, vo, s + far_o);
    }
};

// ------------------------------------------------------------------ operands
// Chunk swizzles of a stage in LDS.  Along the reduction (rows of 128 bytes):
// the 16 lanes of a ds_read_b128 pass, reading one chunk of 16 consecutive
// rows, cover all banks.  Across it (rows of CPR chunks): the four rows of a
// transposing read's 16 lanes fall on different banks; the widest tile's lanes read
// 16 neighbouring chunks of a row and need none.
__device__ __forceinline__ int along(int r, int c) { return c ^ ((r >> 1) & 7); }
template <int CPR>
__device__ __forceinline__ int across(int k, int c)
{
    return CPR >= 32 ? c : CPR == 16 ? c ^ ((k & 3) << 2) : c ^ (((k >> 1) & 1) << 2);
}

// One operand of a tile: R rows (ALONG) or columns (!ALONG) of a stage, loaded
// by NT threads, 16 bytes each.  The base moves on with every stage, so that
// offsets and bounds stay small whatever the operand's size; loads at or past
// the bound read zeros.
//
// PAIR > 0: the rows come in pairs of groups of PAIR, a wave's columns, of which
// the second is taken from base[1]: with SwiGLU the ups of the first's gates.
template <bool ALONG, int R, int NT, int PAIR>
struct Operand {
    static constexpr int NL = R * 128 / 16 / NT;
    static constexpr int CPR = ALONG ? 8 : R / 8;          // 16-byte chunks of an LDS row
    static constexpr int RPL = NT / CPR;                   // LDS rows per load
    static constexpr int HALVES = PAIR >= RPL ? 2 : 1;
    static_assert(NL >= 1 && NT % CPR == 0 && RPL % 4 == 0, "loads of a stage");
    const uint8_t *base[HALVES];
    uint32_t bytes[HALVES];                                // of the stage from its base
    int64_t step;
    uint32_t voff, rstep, pstep;                           // bytes from load to load, and from pair to pair
    int k;                                                 // ALONG: this lane's first reduction value
    int klen, k0;                                          // reduction values, and those before the stage
    uint32_t pitch, width;                                 // !ALONG: bytes of a row, and of its valid columns

    // rows0, rows1: valid rows from p0 and p1 (ALONG); pair: rows of base[0] from pair to pair; cols: valid columns (!ALONG)
    __device__ __forceinline__ void init(const uint16_t *p0, const uint16_t *p1, int rows0, int rows1, int pair, int64_t ld,
                                         int klen_, int64_t cols)
    {
        const int t = threadIdx.x, row = t / CPR;
        base[0] = (const uint8_t *)p0;
        rstep = (uint32_t)(RPL * ld * 2);
        pstep = (uint32_t)(pair * ld * 2);
        klen = klen_;
        k0 = 0;
        if constexpr (ALONG) {
            // up to the stage's end in the last row: what lies past klen there is left to the lanes (lane_offset), and
            // a row after it starts at or past the bound
            const int chunk = along(row, t % CPR);
            const int64_t last = min(ld, (int64_t)kStage);
            bytes[0] = rows0 > 0 ? (uint32_t)((rows0 - 1) * ld + last) * 2 : 0;
            voff = (uint32_t)(row * ld * 2) + chunk * 16;
            if constexpr (HALVES == 2) {
                base[1] = (const uint8_t *)p1;
                bytes[1] = rows1 > 0 ? (uint32_t)((rows1 - 1) * ld + last) * 2 : 0;
            } else if (PAIR > 0) {
                // one load takes both groups, which lie at most 32 rows apart
                static_assert(PAIR == 0 || 2 * PAIR == R || PAIR >= RPL, "a pair in one load");
                const int64_t apart = p1 - p0;
                if (rows1 > 0) bytes[0] = (uint32_t)(apart + (rows1 - 1) * ld + last) * 2;
                if (row >= PAIR) voff = (uint32_t)(apart + (row - PAIR) * ld) * 2 + chunk * 16;
            }
            step = kStage * 2;
            k = chunk * 8;
        } else {
            const int chunk = across<CPR>(row, t % CPR);
            pitch = (uint32_t)ld * 2;
            width = (uint32_t)min(cols, (int64_t)R) * 2;
            voff = row * pitch + (uint32_t)min((int64_t)chunk * 8, cols - 8) * 2;
            step = kStage * ld * 2;
            k = 0;
            bound();
        }
    }
    __device__ __forceinline__ void bound()
    {
        if constexpr (!ALONG) {
            const int rows = min(klen - k0, kStage);
            bytes[0] = rows > 0 ? (uint32_t)(rows - 1) * pitch + width : 0;
        }
    }
    // This lane's offset in the stage, the same for all its loads.
    __device__ __forceinline__ uint32_t lane_offset() const { return !ALONG || k0 + k < klen ? voff : kOOB; }
    // One of the stage's loads into the slot at `lds`, and the step to the next stage after the last.
    __device__ __forceinline__ void issue_one(uint8_t *lds, int i, uint32_t v, int wave) const
    {
        constexpr int LPG = HALVES == 2 ? PAIR / RPL : NL;           // loads of a group
        const int q = i / LPG, h = HALVES == 2 ? q & 1 : 0;
        dma16(base[h], bytes[h], lds + wave * kWave * 16 + i * NT * 16, v, (HALVES == 2 ? (q >> 1) * pstep : 0u) + (i % LPG) * rstep);
    }
    __device__ __forceinline__ void advance()
    {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) base[h] += step;
        k0 += kStage;
        bound();
    }
    __device__ __forceinline__ void issue(uint8_t *lds, int wave)
    {
        const uint32_t v = lane_offset();
#pragma unroll
        for (int i = 0; i < NL; ++i) issue_one(lds, i, v, wave);
        advance();
    }
};

template <int OFF>
__device__ __forceinline__ uintx2 read_tr(uint32_t addr)
{
    uintx2 v;
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
    return v;
}

// Per-lane address in a stage of the fragment of a block of 32 rows / columns from
// `first`: lane l holds row / column l % 32 and reduction values (l / 32) 8 on.
template <bool ALONG, int R>
__device__ __forceinline__ uint32_t frag_base(int first)
{
    const int lane = threadIdx.x & 63, r32 = lane & 31, h = lane >> 5, g16 = (lane >> 4) & 1, s16 = lane & 15;
    if (ALONG) {
        const int sw = (r32 >> 1) & 7;         // chunk 2 j + h of the row is at base ^ (j << 5)
        return (uint32_t)(first + r32) * 128 + (uint32_t)((h ^ sw) & 1) * 16 + (uint32_t)((sw & 6) << 4);
    }
    const int krow = h * 8 + (s16 >> 2), col = first + 16 * g16 + 4 * (s16 & 3);
    return (uint32_t)krow * (R * 2) + (uint32_t)across<R / 8>(krow, col >> 3) * 16 + 8 * (s16 & 1);
}

template <bool ALONG, int R>
struct Frags {
    uint32_t at;
    __device__ __forceinline__ void init(uint32_t lds, int first) { at = lds + frag_base<ALONG, R>(first); }
    template <int KS, int I>
    __device__ __forceinline__ bf16x8 read(uint32_t slot) const
    {
        if constexpr (ALONG) {
            return __builtin_bit_cast(bf16x8, ldsr_u128<I * 32 * 128>((at + slot) ^ (uint32_t)(KS << 5)));
        } else {
            constexpr int O = KS * 16 * R * 2;
            const uint32_t a = (at + slot) ^ (uint32_t)(I << 6);       // a block's 64 bytes: the rows' swizzle moves whole ones
            const uintx2 lo = read_tr<O>(a), hi = read_tr<O + 4 * R * 2>(a);
            return __builtin_bit_cast(bf16x8, uintx4{lo[0], lo[1], hi[0], hi[1]});
        }
    }
};

// Wait for the LDS reads issued so far; the fragments pass through, so that no
// product on them moves before it.
template <int NA, int NB>
__device__ __forceinline__ void wait_frags(bf16x8 (&a)[NA], bf16x8 (&b)[NB])
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < NA; ++i) asm volatile("" : "+v"(a[i]));
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(b[i]));
}
// ------------------------------------------------------------------ kernel
// Bytes of a row of C fp32 sums in LDS: 16 more, so that rows start on other banks.
template <int C>
constexpr int wave_pitch() { return C * 4 + 16; }

// Tile TM x TN by WM x WN waves, times WK that share a stage's four steps of
// the reduction; NS slots of the ring.
template <int TM, int TN, int WM, int WN, int WK, int NS>
struct Shape {
    static constexpr int NT = kWave * WM * WN * WK;
    static constexpr int MI = TM / WM / 32, NJ = TN / WN / 32;
    static constexpr int SLOTA = TM * 128, SLOTB = TN * 128, SLOT = SLOTA + SLOTB, RING = NS * SLOT;
    static constexpr int EPI = 32 * wave_pitch<NJ * 32>() * (WK > 1 ? MI * WK : 1);      // a wave's LDS in the epilogue
    static constexpr int EPIS = WK > 1 ? EPI : EPI * WM * WN;
    static constexpr int LDS = RING > EPIS ? RING : EPIS;
    static_assert(LDS <= (160 << 10) && (WK == 1 || WM * WN == 1), "LDS of a tile");
};

// Logical number of workgroup b of n: consecutive ones share an XCD and its L2.
__device__ __forceinline__ uint32_t xcd_order(uint32_t b, uint32_t n)
{
    const uint32_t q = n / 8, r = n % 8, x = b % 8;
    return x * q + min(x, r) + b / 8;
}

// A wave's sums finished: 32 rows at a time go through the wave's own part of LDS
// in fp32, so that lanes hold 8 neighbouring columns and a row leaves in whole
// lines; nothing waits for another wave.  Lane l holds of a block of 32 x 32 row
// l % 32 and columns (r / 4) 8 + (l / 32) 4 + r % 4, of one of 16 x 16 row l % 16
// and columns (l / 16) 4 + r.  Spread (the widest tile across the reduction), the
// rows and columns of block i are every NJ-th from i on instead: NJ neighbouring
// columns lie in one lane.  With SwiGLU the wave's first C / 2
// columns are gates, the others their ups.  WK waves hold sums of the same outputs:
// they meet in LDS, where each finishes its share of the rows.
template <int PITCH, bool SPREAD, int MI, int NJ>
__device__ __forceinline__ void put_rows(const floatx16 (&acc)[MI][NJ], int i, uint8_t *to)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *(floatx4 *)(to + (lane & 31) * PITCH + (j * 32 + q * 8 + (lane >> 5) * 4) * 4) =
                floatx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
}
template <int PITCH, bool SPREAD, int MI, int NJ>
__device__ __forceinline__ void put_rows(const floatx4 (&acc)[MI][NJ], int i, uint8_t *to)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint8_t *row = to + (h * 16 + (lane & 15)) * PITCH;
        if constexpr (SPREAD) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < NJ; j += 4) {
                    floatx4 v;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float f;
                        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(f) : "a"(acc[2 * i + h][j + x][r]));
                        v[x] = f;
                    }
                    *(floatx4 *)(row + (((lane >> 4) * 4 + r) * NJ + j) * 4) = v;
                }
        } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j) *(floatx4 *)(row + (j * 16 + (lane >> 4) * 4) * 4) = acc[2 * i + h][j];
        }
    }
}

template <int FIN, bool F32, int MI, int NJ, int WK, bool SPREAD_M, bool SPREAD_N, class Acc>
__device__ __forceinline__ void finish_wave_as(const LinearParams &p, const Acc &acc, uint8_t *lds, int wk, int64_t m0,
                                               int64_t n0, float *partial, int64_t ldp)
{
    constexpr int C = NJ * 32, PITCH = wave_pitch<C>();
    constexpr bool GLU = FIN == kFinFwdGlu;
    constexpr int GROUPS = C / (GLU ? 16 : 8), RPI = 64 / GROUPS;      // lanes of a row, rows of an instruction
    constexpr int ROWS = WK > 1 ? MI * 32 / WK : 32, ITS = (ROWS + RPI - 1) / RPI;
    const int lane = threadIdx.x & 63, g = lane % GROUPS, r0 = lane / GROUPS;
    const int64_t n = n0 + g * 8, ncols = GLU ? p.N >> 1 : p.N;
    // from a place in the order of LDS's rows to the row of the product; a lane's first is its r0 or, spread, 8 r0
    static_assert(!SPREAD_M || (RPI == 4 && MI == 4), "rows of a spread block");
    const int first = SPREAD_M ? 8 * r0 : r0;
    auto row_of = [&](int at) { return SPREAD_M ? (at & 15) * 8 + (at >> 5) * 2 + (at >> 4 & 1) : at; };
    auto get = [&](const uint8_t *src, float (&v)[8]) {
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const floatx4 a = *(const floatx4 *)(src + w * MI * 32 * PITCH), b = *(const floatx4 *)(src + w * MI * 32 * PITCH + 16);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                v[x] = w ? v[x] + a[x] : a[x];
                v[4 + x] = w ? v[4 + x] + b[x] : b[x];
            }
        }
    };
    // rows of LDS from `from` on; the next row's loads go out before one is worked on, in pairs that take each other's
    // registers.  Loops, not copies: a wide tile's all unrolled were 350 KB of code that each workgroup had to fetch
    auto share = [&](auto &&put_row, int from) {
        const uint8_t *src = lds + (from + r0) * PITCH + g * 32;
        float v0[8], u0[8], v1[8], u1[8];
        auto next = [&](int it, float (&v)[8], float (&u)[8]) {
            const uint8_t *s = src + min(it, ITS - 1) * RPI * PITCH;
            get(s, v);
            if (GLU) get(s + C / 2 * 4, u);
        };
        next(0, v0, u0);
        if constexpr (ITS == 1) {
            put_row(IC<0>{}, 0, v0, u0);
        } else {
            static_assert(ITS % 2 == 0, "rows in pairs");
#pragma unroll 1
            for (int it = 0; it < ITS; it += 2) {
                next(it + 1, v1, u1);
                put_row(IC<0>{}, it, v0, u0);
                next(it + 2, v0, u0);
                put_row(IC<1>{}, it + 1, v1, u1);
            }
        }
    };
    auto all = [&](auto &&put_row) {
        if constexpr (WK > 1) {
#pragma unroll
            for (int i = 0; i < MI; ++i) put_rows<PITCH, SPREAD_N>(acc, i, lds + (wk * MI + i) * 32 * PITCH);
            __syncthreads();
            if (r0 < ROWS) share([&](auto P, int it, float (&v)[8], float (&u)[8]) { put_row(P, wk * ROWS + it * RPI, v, u); }, wk * ROWS);
        } else {
#pragma unroll 1
            for (int i = 0; i < MI; ++i) {
                unrolled<MI>([&](auto I) {
                    if (i == I.value) {
                        put_rows<PITCH, SPREAD_N>(acc, I.value, lds);
                        asm volatile("; rows %0" ::"i"(I.value) : "memory");   // the cases stay apart: registers have no index
                    }
                });
                asm volatile("" ::: "memory");         // lanes read what others wrote: LDS keeps a wave's order
                share([&](auto P, int it, float (&v)[8], float (&u)[8]) { put_row(P, i * 32 + it * RPI, v, u); }, 0);
                asm volatile("" ::: "memory");
            }
        }
    };
    if (m0 >= p.M && WK == 1) return;
    if constexpr (FIN == kFinPartial) {
        const uint8_t *out = (const uint8_t *)partial;
        const uint32_t row_b = (uint32_t)ldp * 4, bytes = (uint32_t)max(min(p.M - m0, (int64_t)kWideRows), (int64_t)0) * row_b;
        const uint32_t vo = n < ldp ? first * row_b + (uint32_t)n * 4 : kOOB;
        all([&](auto, int at, float (&v)[8], float (&)[8]) {
            const int row = row_of(at);
            buf_store(uintx4{f32_bits(v[0]), f32_bits(v[1]), f32_bits(v[2]), f32_bits(v[3])}, out, bytes, vo, row * row_b);
            buf_store(uintx4{f32_bits(v[4]), f32_bits(v[5]), f32_bits(v[6]), f32_bits(v[7])}, out, bytes, vo, row * row_b + 16);
        });
    } else {
        const FinishRows<FIN, F32> fin(p.f, m0, p.M, first, n, n < ncols);
        Extra x[2] = {};
        fin.fetch(x[0], WK > 1 ? wk * ROWS : 0);
        all([&](auto P, int at, float (&v)[8], float (&u)[8]) {
            constexpr int I = decltype(P)::value;
            if (ITS > 1) fin.fetch(x[1 - I], row_of(at + RPI));
            fin.store(x[I], row_of(at), v, u);
        });
    }
}

// OP: the operator, which says what there is to finish.  in_parts: the sums are those
// of a part of the reduction, and go to `partial`, the wave's first row there, whose
// rows are ldp apart, from column n0 on.
template <int OP, int MI, int NJ, int WK, bool SPREAD_M = false, bool SPREAD_N = false, class Acc>
__device__ __forceinline__ void finish_wave(const LinearParams &p, const Acc &acc, uint8_t *lds, int wk, int64_t m0,
                                            int64_t n0, bool in_parts, float *partial, int64_t ldp)
{
    constexpr int PLAIN = OP == kLinDgrad ? kFinGrad : kFinFwd, GLU = OP == kLinDgrad ? kFinGradGlu : kFinFwdGlu;
    auto as = [&](auto F, auto F32) {
        finish_wave_as<decltype(F)::value, decltype(F32)::value, MI, NJ, WK, SPREAD_M, SPREAD_N>(p, acc, lds, wk, m0, n0, partial, ldp);
    };
    if (in_parts) return as(IC<kFinPartial>{}, IC<true>{});
    if constexpr (OP == kLinWgrad) {
        as(IC<PLAIN>{}, IC<true>{});
    } else if (p.f.finish == GLU) {
        if (OP == kLinFwd && p.f.f32) as(IC<GLU>{}, IC<OP == kLinFwd>{});
        else as(IC<GLU>{}, IC<false>{});
    } else if (OP == kLinFwd && p.f.f32) {
        as(IC<PLAIN>{}, IC<OP == kLinFwd>{});
    } else {
        as(IC<PLAIN>{}, IC<false>{});
    }
}

// A workgroup's place in the product: its tile, its part of the reduction and the
// operands' loads.
template <bool ALA, bool ALB, int TM, int TN, int NT, int C>
struct Place {
    int64_t m0, n0;
    int klen;
    bool glu;
    Operand<ALA, TM, NT, 0> a;
    Operand<ALB, TN, NT, ALB ? C / 2 : 0> b;             // a wave has C columns

    // reduction values kb on, klen at most
    __device__ __forceinline__ void init(const LinearParams &p, int tile, int tilesM, int tilesN, int64_t kb, int64_t len)
    {
        int mt, nt;
        grouped_tile_order(tile, tilesM, tilesN, mt, nt);
        m0 = (int64_t)mt * TM;
        glu = p.f.finish == kFinFwdGlu;
        klen = (int)min(p.K - kb, len);
        // columns of the tile: n0 on; with SwiGLU, half as many gates and their ups, C / 2 of each to a wave
        n0 = (int64_t)nt * (glu ? TN / 2 : TN);
        const int64_t half = p.N >> 1;
        const int rows = (int)min(p.M - m0, (int64_t)TM);
        if (ALA) a.init(p.a + m0 * p.lda + kb, nullptr, rows, 0, 0, p.lda, klen, 0);
        else a.init(p.a + kb * p.lda + m0, nullptr, 0, 0, 0, p.lda, klen, p.M - m0);
        if (ALB) {
            const int64_t n1 = glu ? half + n0 : n0 + C / 2;
            const int rows0 = (int)min((glu ? half : p.N) - n0, (int64_t)(glu ? TN / 2 : TN));
            b.init(p.b + n0 * p.ldb + kb, p.b + n1 * p.ldb + kb, rows0, glu ? rows0 : rows0 - C / 2, glu ? C / 2 : C, p.ldb, klen, 0);
        } else {
            b.init(p.b + kb * p.ldb + n0, nullptr, 0, 0, 0, p.ldb, klen, p.N - n0);
        }
    }
    // first column of wave wn's outputs
    __device__ __forceinline__ int64_t col(int wn) const { return n0 + wn * (glu ? C / 2 : C); }
};

template <bool ALA, bool ALB, int TM, int TN, int WM, int WN, int WK, int NS>
__global__ __launch_bounds__(64 * WM * WN * WK, 2) void linear_kernel(LinearParams p, int tilesM, int tilesN)
{
    using S = Shape<TM, TN, WM, WN, WK, NS>;
    constexpr int NT = S::NT, MI = S::MI, NJ = S::NJ;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / WK / WN;

    const uint32_t id = xcd_order(blockIdx.x, gridDim.x), tiles = (uint32_t)tilesM * (uint32_t)tilesN;
    const int64_t split = id / tiles;
    Place<ALA, ALB, TM, TN, NT, NJ * 32> at;
    at.init(p, (int)(id % tiles), tilesM, tilesN, split * p.part, p.part);
    const uint32_t lds0 = lds_addr(smem);
    Frags<ALA, TM> ra;
    Frags<ALB, TN> rb;
    ra.init(lds0, wm * MI * 32);
    rb.init(lds0 + S::SLOTA, wn * NJ * 32);
    static_assert(WK == 1 || (ALA && ALB), "waves that share a stage's steps read along the reduction");
    if (WK > 1) ra.at ^= (uint32_t)wk << 5, rb.at ^= (uint32_t)wk << 5;      // the wave's own step

    floatx16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    constexpr int LA = decltype(at.a)::NL, L = LA + decltype(at.b)::NL;       // loads of a stage
    const int nk = (at.klen + kStage - 1) / kStage;
    auto issue = [&](int slot) {
        at.a.issue(smem + slot * S::SLOT, wave);
        at.b.issue(smem + slot * S::SLOT + S::SLOTA, wave);
    };
    // stages past the end load zeros, so that the waits need no cases
    if constexpr (WK == 1) {
        // A stage's fragments are read while the one before is multiplied, so that LDS's latency is paid once a stage and
        // the slot is free again as soon as all waves hold them: NS stages are under way beside the one in registers
        bf16x8 fa[2][4][MI], fb[2][4][NJ];
        constexpr int P = 4 * MI * NJ, R = 4 * (MI + NJ);    // products and reads of a stage
#pragma unroll
        for (int st = 0; st < NS; ++st) issue(st);
        wait_vmcnt<(NS - 1) * L>();
        barrier();
        unrolled<4>([&](auto KS) {
            unrolled<MI>([&](auto I) { fa[0][KS.value][I.value] = ra.template read<KS.value, I.value>(0); });
            unrolled<NJ>([&](auto I) { fb[0][KS.value][I.value] = rb.template read<KS.value, I.value>(0); });
        });
        unrolled<4>([&](auto KS) { wait_frags(fa[0][KS.value], fb[0][KS.value]); });
        uint32_t slot = 0, next = NS == 1 ? 0 : S::SLOT;
        auto stage = [&](auto CC) {
            constexpr int C = decltype(CC)::value;
            wait_vmcnt<(NS - 2) * L>();              // the next stage has landed for this wave, and after the barrier for all
            barrier();
            const uint32_t va = at.a.lane_offset(), vb = at.b.lane_offset();
            unrolled<P>([&](auto X) {
                constexpr int x = decltype(X)::value, ks = x / (MI * NJ), i = x / NJ % MI, j = x % NJ;
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[C][ks][j], fa[C][ks][i], acc[i][j], 0, 0, 0);
                unrolled<(x + 1) * R / P - x * R / P>([&](auto Y) {
                    constexpr int y = x * R / P + decltype(Y)::value, k = y / (MI + NJ), q = y % (MI + NJ);
                    if constexpr (q < MI) fa[1 - C][k][q] = ra.template read<k, q>(next);
                    else fb[1 - C][k][q - MI] = rb.template read<k, q - MI>(next);
                });
                unrolled<(x + 1) * L / P - x * L / P>([&](auto Y) {
                    constexpr int y = x * L / P + decltype(Y)::value;
                    if constexpr (y < LA) at.a.issue_one(smem + slot, y, va, wave);
                    else at.b.issue_one(smem + slot + S::SLOTA, y - LA, vb, wave);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            at.a.advance();
            at.b.advance();
            unrolled<4>([&](auto KS) { wait_frags(fa[1 - C][KS.value], fb[1 - C][KS.value]); });
            slot = next;
            next = next == (NS - 1) * S::SLOT ? 0 : next + S::SLOT;
        };
        int kt = 0;
        for (; kt + 2 <= nk; kt += 2) {
            stage(IC<0>{});
            stage(IC<1>{});
        }
        if (kt < nk) stage(IC<0>{});
    } else {
        static_assert(WK == 4, "a step of the stage per wave");
#pragma unroll
        for (int st = 0; st < NS - 1; ++st) issue(st);
        bf16x8 fa[MI], fb[NJ];
        int slot = 0;
        for (int kt = 0; kt < nk; ++kt) {
            wait_vmcnt<(NS - 2) * L>();
            barrier();
            const uint32_t so = (uint32_t)slot * S::SLOT;
            unrolled<MI>([&](auto I) { fa[I.value] = ra.template read<0, I.value>(so); });
            unrolled<NJ>([&](auto I) { fb[I.value] = rb.template read<0, I.value>(so); });
            wait_frags(fa, fb);
            issue(slot == 0 ? NS - 1 : slot - 1);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
            slot = slot + 1 == NS ? 0 : slot + 1;
        }
    }
    wait_vmcnt<0>();                             // zeros of stages past the end may still be landing in the ring
    barrier();

    const int64_t m0 = at.m0 + wm * MI * 32;
    finish_wave<ALA ? ALB ? kLinFwd : kLinDgrad : kLinWgrad, MI, NJ, WK>(p, acc, smem + (WK > 1 ? 0 : wave * S::EPI), wk, m0, at.col(wn), p.splits > 1,
                                                                         p.partials + (split * p.M + m0) * p.N, p.N);
}

// ------------------------------------------------------------------ wide tile
// The tile for products that fill the chip: 256 x 256 by four waves of 128 x 128,
// one on each SIMD, with 256 accumulators each.  A wave's share is square because
// LDS is the narrow place: the waves read 128 KB of a stage here, eight waves of
// 128 x 64 would read 192 KB, which with the 64 KB that the loads bring in takes
// LDS as long as the products take the matrix cores (8192^3: 1060 TFLOP/s so).
//
// One wave a SIMD hides nothing by itself, so the order of its instructions does.
// A stage is two steps of 32 reduction values, 64 products of 16 x 16 x 32 each.
// While a step's run, the next one's fragments are read, one read every second or
// third product, and eight loads go out, one every eighth: in one go either holds
// the products up (3169 cycles a stage, spread 2371, the products alone 2048).
// 16 x 16 x 32 because at the power limit it gets the same work done in 1.32 us a
// stage that 32 x 32 x 16 does in 1.41.
//
// LDS holds three slots of A and two of B, all of its 160 KB.  Step 0 of stage t
// loads A of t + 2, step 1 B of t + 2 into the slot that B of t has left.  The one
// barrier of a stage stands between its steps: stage t's fragments are all in
// registers by then, and all loads but those of A of t + 2 have landed.
constexpr int kWideThreads = 256, kWideSlot = kWide * 128, kWideLds = 5 * kWideSlot;

// A wave's eight fragments of one operand at step KS (32 values) of a stage.  Along
// the reduction fragment i holds 16 rows from 16 i on, lane l row l % 16 and
// reduction values (l / 16) 8 on: a read each.  Across it a lane reads eight
// neighbouring columns, from 8 (l % 16) on, at each of its eight reduction values,
// and turns the 8 x 8 block itself, a v_perm_b32 a register: fragment i then holds
// of lane l column 8 (l % 16) + i.  (The transposing LDS reads need no turning but
// take LDS half as long again, which it has not got here: wgrad 2818 cycles a stage.)
template <bool ALONG>
struct WideFrags {
    uint32_t at;
    __device__ __forceinline__ void init(uint32_t lds, int first)
    {
        const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
        if (ALONG) at = lds + (uint32_t)(first + r16) * 128 + (uint32_t)along(first + r16, q) * 16;
        else at = lds + (uint32_t)(q * 8 * kWide + first + r16 * 8) * 2;
    }
    template <int KS, int I>
    __device__ __forceinline__ uintx4 read(uint32_t slot) const
    {
        if constexpr (ALONG) return ldsr_u128<I * 16 * 128>((at + slot) ^ (uint32_t)(KS << 6));     // chunk q + 4 KS
        else return ldsr_u128<(KS * 32 + I) * kWide * 2>(at + slot);
    }
    // word W of fragment I
    template <int I, int W>
    static __device__ __forceinline__ uint32_t turned(const uintx4 (&raw)[8])
    {
        return __builtin_amdgcn_perm(raw[2 * W + 1][I / 2], raw[2 * W][I / 2], I & 1 ? 0x07060302u : 0x05040100u);
    }
};

// The LDS reads but the last N have arrived; what they brought passes through, so
// that no use of it moves before.
template <int N>
__device__ __forceinline__ void wait_reads(uintx4 (&v)[8])
{
    asm volatile("s_waitcnt lgkmcnt(%0)" ::"i"(N) : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(v[i]));
}

template <bool ALA, bool ALB>
__global__ __launch_bounds__(kWideThreads, 1) void linear_wide_kernel(LinearParams p, int tilesM, int tilesN)
{
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wm = wave >> 1;
    // this workgroup's piece of the work
    const WideCut &cut = p.cut;
    const int rest = cut.rest, left = rest - cut.tails, mains = cut.parts * rest;
    int b = blockIdx.x, tile, slot = -1;
    int64_t kb = 0, len = p.K;
    if (b < cut.whole) {
        tile = xcd_order(b, cut.whole);
    } else if ((b -= cut.whole) < mains) {
        slot = xcd_order(b, mains);
        tile = cut.whole + slot % rest;
        kb = slot / rest * cut.main;
        len = cut.main;
    } else if ((b -= mains) < cut.tails) {
        const int t = xcd_order(b, cut.tails);
        slot = mains + t;
        tile = cut.whole + t;
        kb = cut.parts * cut.main;
    } else {
        const int t = xcd_order(b - cut.tails, left * cut.cuts);
        slot = mains + cut.tails + t;
        tile = cut.whole + cut.tails + t % left;
        kb = cut.parts * cut.main + t / left * cut.cut;
        len = cut.cut;
    }
    Place<ALA, ALB, kWide, kWide, kWideThreads, 128> at;
    at.init(p, tile, tilesM, tilesN, kb, len);
    const uint32_t lds0 = lds_addr(smem);
    uint8_t *const smem_b = smem + 3 * kWideSlot;
    WideFrags<ALA> ra;
    WideFrags<ALB> rb;
    ra.init(lds0, wm * 128);
    rb.init(lds0 + 3 * kWideSlot, wn * 128);
    floatx4 acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = floatx4{0, 0, 0, 0};
    constexpr int NL = kWideSlot / 16 / kWideThreads;        // loads of an operand's stage
    static_assert(NL == 8, "eight loads a step");
    const int nk = (at.klen + kStage - 1) / kStage;
    at.a.issue(smem, wave);
    at.b.issue(smem_b, wave);
    at.a.issue(smem + kWideSlot, wave);
    at.b.issue(smem_b + kWideSlot, wave);
    if (at.m0 + wm * 128 >= p.M || at.col(wn) >= (at.glu ? p.N >> 1 : p.N)) {
        // nothing of this wave's share is in the matrix: it loads, and keeps the others' barriers (2880 columns are 11.25
        // tiles: the power that its products would take lets the clock rise, 251 to 244 us for 16384 x 2880 x 2880 wgrad)
        wait_vmcnt<2 * NL>();
        barrier();
        int sa = 2 * kWideSlot, sb = 0;
        for (int kt = 0; kt < nk; ++kt) {
            at.a.issue(smem + sa, wave);
            wait_vmcnt<NL>();
            barrier();
            at.b.issue(smem_b + sb, wave);
            sa = sa == 2 * kWideSlot ? 0 : sa + kWideSlot;
            sb = kWideSlot - sb;
        }
        wait_vmcnt<0>();
        barrier();
        return;
    }
    uintx4 fa[2][8], fb[2][8];
    // word W of fragment I out of what was read
    auto turn = [&](auto ALONG, uintx4 (&f)[8], const uintx4 (&raw)[8], auto IW) {
        constexpr int I = decltype(IW)::value / 4, W = decltype(IW)::value % 4;
        if constexpr (!decltype(ALONG)::value) f[I][W] = WideFrags<false>::turned<I, W>(raw);
        else if constexpr (W == 0) f[I] = raw[I];
    };
    using AlongA = IC<ALA>;
    using AlongB = IC<ALB>;
    wait_vmcnt<2 * NL>();
    barrier();
    {
        uintx4 xa[8], xb[8];
        unrolled<8>([&](auto I) { xa[I.value] = ra.template read<0, I.value>(0); });
        unrolled<8>([&](auto I) { xb[I.value] = rb.template read<0, I.value>(0); });
        wait_reads<0>(xa);
        wait_reads<0>(xb);
        unrolled<32>([&](auto IW) { turn(AlongA{}, fa[0], xa, IW); });
        unrolled<32>([&](auto IW) { turn(AlongB{}, fb[0], xb, IW); });
    }

    uint32_t a0 = 0, a1 = kWideSlot, a2 = 2 * kWideSlot, b0 = 0, b1 = kWideSlot;     // slots of this stage and the next ones
    auto step = [&](auto KC) {
        constexpr int KS = decltype(KC)::value, C = KS, NKS = 1 - KS;
        const uint32_t sa = KS ? a1 : a0, sb = KS ? b1 : b0;                         // where the next step's fragments are
        const uint32_t v = KS ? at.b.lane_offset() : at.a.lane_offset();
        // reads every READ products: across the reduction the last of them turn what was read
        constexpr int READ = ALA && ALB ? 3 : 2;
        uintx4 xa[8], xb[8];
        unrolled<64>([&](auto X) {
            constexpr int x = decltype(X)::value, i = x >> 3, j = x & 7;
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[C][j]), __builtin_bit_cast(bf16x8, fa[C][i]),
                                                                acc[i][j], 0, 0, 0);
            if constexpr (x % READ == 0 && x < 16 * READ) {
                constexpr int y = x / READ;
                if constexpr (y < 8) xb[y] = rb.template read<NKS, y>(sb);
                else xa[y - 8] = ra.template read<NKS, y - 8>(sa);
            }
            if constexpr (x % 8 == 4) {
                if constexpr (KS == 0) at.a.issue_one(smem + a2, x / 8, v, wave);
                else at.b.issue_one(smem_b + b0, x / 8, v, wave);
            }
            if constexpr (!ALB) {
                constexpr int T = ALA ? 1 : 2, FROM = 32;
                if constexpr (x == FROM) wait_reads<8>(xb);
                if constexpr (x >= FROM && x < FROM + 32 / T)
                    unrolled<T>([&](auto Y) { turn(AlongB{}, fb[1 - C], xb, IC<(x - FROM) * T + decltype(Y)::value>{}); });
            }
            if constexpr (!ALA) {
                if constexpr (x == 48) wait_reads<0>(xa);
                if constexpr (x >= 48) unrolled<2>([&](auto Y) { turn(AlongA{}, fa[1 - C], xa, IC<(x - 48) * 2 + decltype(Y)::value>{}); });
            }
            if constexpr (x % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (KS == 0) at.a.advance();
        else at.b.advance();
        if constexpr (ALA) {
            wait_reads<0>(xa);
            unrolled<8>([&](auto I) { fa[1 - C][I.value] = xa[I.value]; });
        }
        if constexpr (ALB) {
            wait_reads<0>(xb);
            unrolled<8>([&](auto I) { fb[1 - C][I.value] = xb[I.value]; });
        }
        if constexpr (KS == 0) {
            wait_vmcnt<NL>();            // all but A of the stage after next has landed, for all waves after the barrier
            barrier();
        }
    };
    for (int kt = 0; kt < nk; ++kt) {
        step(IC<0>{});
        step(IC<1>{});
        const uint32_t a = a0;
        a0 = a1;
        a1 = a2;
        a2 = a;
        b1 = b0;
        b0 = kWideSlot - b1;
    }
    wait_vmcnt<0>();                     // zeros of stages past the end may still be landing in the ring
    barrier();
    // across the reduction the epilogue reads the sums by instructions of its own, which wait for no product: 32 states
    // after the loop's last one
    if constexpr (!ALB) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    // a piece's sums go to a tile of their own, its columns in the waves' order
    finish_wave<ALA ? ALB ? kLinFwd : kLinDgrad : kLinWgrad, 4, 4, 1, !ALA, !ALB>(p, acc, smem + wave * 32 * wave_pitch<128>(), 0, at.m0 + wm * 128,
                                                                     slot < 0 ? at.col(wn) : wn * 128, slot >= 0,
                                                                     p.partials + ((int64_t)slot * kWide + wm * 128) * kWide, kWide);
}

// The parts' column sums added in order, a column to a thread.  Where a product's
// parts are joined too, the same launch does both.
__device__ __forceinline__ void colsum_join(const ColsumParams &p, int block)
{
    const int64_t c = (int64_t)block * kThreads + threadIdx.x;
    if (c >= p.N) return;
    float sum = 0.0f;
#pragma unroll 8
    for (int i = 0; i < p.parts; ++i) sum += p.partials[(int64_t)i * p.N + c];
    p.dbias[c] = p.accumulate ? p.dbias[c] + sum : sum;
}

// The pieces of a cut tile added in their order along the reduction, then what the
// tile itself would have done.  A workgroup takes 8 rows (SwiGLU: 16), a thread 8 columns.
template <int FIN>
__global__ __launch_bounds__(kThreads) void linear_wide_join_kernel(LinearParams p, int tilesM, int tilesN)
{
    constexpr bool GLU = FIN == kFinFwdGlu;
    constexpr int GROUPS = kWide / (GLU ? 16 : 8), ROWS = kThreads / GROUPS;
    if (FIN == kFinFwd && (int)blockIdx.x >= p.join_blocks) return colsum_join(p.sums, (int)blockIdx.x - p.join_blocks);
    const WideCut &cut = p.cut;
    const int t = blockIdx.x / (kWide / ROWS), g = threadIdx.x % GROUPS;
    const int row = blockIdx.x % (kWide / ROWS) * ROWS + (int)threadIdx.x / GROUPS;
    int mt, nt;
    grouped_tile_order(cut.whole + t, tilesM, tilesN, mt, nt);
    const int64_t m = (int64_t)mt * kWide + row, n = (int64_t)nt * (GLU ? kWide / 2 : kWide) + g * 8;
    if (m >= p.M || n >= (GLU ? p.N >> 1 : p.N)) return;
    // a wave's 128 columns are 64 gates and their ups
    const float *src = p.partials + row * kWide + (GLU ? g / 8 * 128 + g % 8 * 8 : g * 8);
    float v[8] = {}, u[8] = {};
    auto add = [&](int slot) {
        float f[8];
        load_stream<true, false>(src, (int64_t)slot * kWide * kWide, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[j];
        if (GLU) {
            load_stream<true, false>(src, (int64_t)slot * kWide * kWide + 64, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] += f[j];
        }
    };
    const int mains = cut.parts * cut.rest;
#pragma unroll 4
    for (int i = 0; i < cut.parts; ++i) add(i * cut.rest + t);
    if (t < cut.tails) {
        add(mains + t);
    } else {
        const int left = cut.rest - cut.tails;
#pragma unroll 4
        for (int i = 0; i < cut.cuts; ++i) add(mains + cut.tails + i * left + t - cut.tails);
    }
    finish_row<FIN>(p.f, m, n, v, u);
}

// ------------------------------------------------------------------ few rows
// At most 16 rows against w [N, K]: w is read once, x comes from L2.  A
// workgroup takes 16 columns (8 gates and their ups), its eight waves the
// steps of 64 reduction values in turn: a wave's loads of a step are whole
// lines of 16 rows.  The reduction's values are taken in the order in which a
// lane's two 16-byte loads find them, alike for both operands.  The waves'
// sums meet in LDS and are added in order.
constexpr int kFewWaves = 8, kFewCols = 16;

__global__ __launch_bounds__(kFewWaves * kWave) void linear_few_kernel(LinearParams p)
{
    constexpr int U = 4;                                     // steps of a batch; two batches are in flight
    constexpr int PITCH = kFewCols + 4;
    __shared__ __attribute__((aligned(16))) float red[kFewWaves][16][PITCH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const bool glu = p.f.finish == kFinFwdGlu;
    const int64_t half = p.N >> 1;
    const int64_t n0 = (int64_t)blockIdx.x * (glu ? kFewCols / 2 : kFewCols);
    int64_t n = glu && r16 >= 8 ? half + n0 + r16 - 8 : n0 + r16;
    if (n >= p.N) n = p.N - 1;                               // read, never stored
    const uint16_t *w = p.b + n * p.ldb + q * 16;
    const uint16_t *x = p.a + min((int64_t)r16, p.M - 1) * p.lda + q * 16;
    floatx4 acc = {0, 0, 0, 0};

    struct Batch {
        uintx4 w[U][2], x[U][2];
    };
    const int K = (int)p.K, full = K / 64;
    auto load = [&](Batch &b, int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // past the end: the last step again, not used
            const int s = min(s0 + u * kFewWaves, full - 1) * 64;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                b.w[u][h] = *(const uintx4 *)(w + s + h * 8);
                b.x[u][h] = *(const uintx4 *)(x + s + h * 8);
            }
        }
    };
    auto mma = [&](const uintx4 &wv, const uintx4 &xv) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv), __builtin_bit_cast(bf16x8, xv), acc, 0, 0, 0);
    };
    auto use = [&](const Batch &b, int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u * kFewWaves >= full) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) mma(b.w[u][h], b.x[u][h]);
        }
    };
    if (wave < full) {
        Batch b0, b1;
        load(b0, wave);
        for (int s = wave; s < full; s += 2 * U * kFewWaves) {
            load(b1, s + U * kFewWaves);
            use(b0, s);
            load(b0, s + 2 * U * kFewWaves);
            use(b1, s + U * kFewWaves);
        }
    }
    // the last K % 64 values, zeros past the end on both sides
    if (K % 64 && wave == full % kFewWaves) {
        const int s = full * 64;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool ok = s + q * 16 + h * 8 < K;
            const int o = ok ? s + h * 8 : -q * 16;          // a lane past the end reads its row's start
            uintx4 wv = *(const uintx4 *)(w + o), xv = *(const uintx4 *)(x + o);
            wv = ok ? wv : uintx4{0, 0, 0, 0};
            xv = ok ? xv : uintx4{0, 0, 0, 0};
            mma(wv, xv);
        }
    }
    // lane l: row l % 16 of x, columns (l / 16) 4 + r
    *(floatx4 *)&red[wave][r16][q * 4] = acc;
    __syncthreads();
    // a thread of the first waves finishes 8 columns of a row
    const int groups = glu ? 1 : 2, m = threadIdx.x / groups, g = threadIdx.x % groups;
    const int64_t nn = n0 + g * 8;
    if (m >= p.M || (!glu && nn >= p.N)) return;
    float v[8] = {}, u[8] = {};
#pragma unroll
    for (int wv = 0; wv < kFewWaves; ++wv)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] += red[wv][m][g * 8 + j];
            if (glu) u[j] += red[wv][m][8 + j];
        }
    if (glu) finish_row<kFinFwdGlu>(p.f, m, nn, v, u);
    else finish_row<kFinFwd>(p.f, m, nn, v, u);
}

// The parts' sums added in order, then what the tile itself would have done.
template <int FIN>
__global__ __launch_bounds__(kThreads) void linear_join_kernel(LinearParams p)
{
    constexpr bool GLU = FIN == kFinFwdGlu;
    if (FIN == kFinFwd && (int)blockIdx.x >= p.join_blocks) return colsum_join(p.sums, (int)blockIdx.x - p.join_blocks);
    const int64_t half = p.N >> 1, groups = (GLU ? half : p.N) / 8, total = p.M * groups;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)p.join_blocks * kThreads) {
        const int64_t m = i / groups, n = (i - m * groups) * 8;
        float v[8] = {}, u[8] = {};
#pragma unroll 8
        for (int s = 0; s < p.splits; ++s) {
            float f[8];
            const int64_t at = (s * p.M + m) * p.N + n;
            load_stream<true, false>(p.partials, at, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += f[j];
            if (GLU) {
                load_stream<true, false>(p.partials, at + half, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] += f[j];
            }
        }
        finish_row<FIN>(p.f, m, n, v, u);
    }
}

// ------------------------------------------------------------------ column sums
// A workgroup adds 64 columns over one part of the rows: 8 lanes of 8 columns,
// 32 rows side by side, joined in LDS in their order.
constexpr int kColsumCols = 64, kColsumRows = 32;
__global__ __launch_bounds__(kThreads) void colsum_kernel(ColsumParams p)
{
    const int64_t M = p.M, N = p.N;
    __shared__ float s[kColsumRows][kColsumCols + 4];
    const int lane = threadIdx.x & 7, side = threadIdx.x >> 3;
    const int64_t n = (int64_t)blockIdx.x * kColsumCols + lane * 8;
    float v[8] = {};
    if (n < N) {
#pragma unroll 4
        for (int64_t r = (int64_t)blockIdx.y * kColsumRows + side; r < M; r += (int64_t)gridDim.y * kColsumRows) {
            float f[8];
            unpack8(*(const uintx4 *)(p.dy + r * N + n), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += f[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[side][lane * 8 + j] = v[j];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * kColsumCols + threadIdx.x;
    if (threadIdx.x >= kColsumCols || c >= N) return;
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < kColsumRows; ++r) sum += s[r][threadIdx.x];
    if (p.parts > 1) p.partials[(int64_t)blockIdx.y * N + c] = sum;
    else p.dbias[c] = p.accumulate ? p.dbias[c] + sum : sum;
}

__global__ __launch_bounds__(kThreads) void colsum_join_kernel(ColsumParams p) { colsum_join(p, blockIdx.x); }

template <int FIN>
__global__ __launch_bounds__(kThreads) void act_bwd_kernel(const uint16_t *dout, FinishParams f, int64_t M)
{
    const int64_t groups = f.N / 8, total = M * groups;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t m = i / groups, n = (i - m * groups) * 8;
        float v[8], u[8];
        unpack8(*(const uintx4 *)(dout + m * f.N + n), v);
        finish_row<FIN>(f, m, n, v, u);
    }
}

// ------------------------------------------------------------------ plan and launch
// Workgroups that join the parts of the column sums.
int sums_join_blocks(const LinearParams &p)
{
    return p.sums.dbias && p.sums.parts > 1 ? (int)((p.sums.N + kThreads - 1) / kThreads) : 0;
}

template <bool ALA, bool ALB, int TM, int TN, int WM, int WN, int WK, int NS>
hipError_t launch_tile(const LinearParams &p, hipStream_t s)
{
    using S = Shape<TM, TN, WM, WN, WK, NS>;
    auto kern = linear_kernel<ALA, ALB, TM, TN, WM, WN, WK, NS>;
    static LdsLimit lds_limit;
    const hipError_t e = lds_limit.ensure((const void *)kern, S::LDS);
    if (e != hipSuccess) return e;
    const int tn = p.f.finish == kFinFwdGlu ? TN / 2 : TN;
    const int64_t cols = p.f.finish == kFinFwdGlu ? p.N / 2 : p.N;
    const int64_t tilesM = (p.M + TM - 1) / TM, tilesN = (cols + tn - 1) / tn, grid = tilesM * tilesN * p.splits;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(S::NT), S::LDS, s, p, (int)tilesM, (int)tilesN);
    return hipGetLastError();
}

template <bool ALA, bool ALB>
hipError_t launch_wide(const LinearParams &p, hipStream_t s)
{
    auto kern = linear_wide_kernel<ALA, ALB>;
    static LdsLimit lds_limit;
    const hipError_t e = lds_limit.ensure((const void *)kern, kWideLds);
    if (e != hipSuccess) return e;
    const bool glu = p.f.finish == kFinFwdGlu;
    const int64_t cols = glu ? p.N / 2 : p.N, tn = glu ? kWide / 2 : kWide;
    const int tilesM = (int)((p.M + kWide - 1) / kWide), tilesN = (int)((cols + tn - 1) / tn);
    hipLaunchKernelGGL(kern, dim3((unsigned)(p.cut.whole + p.cut.pieces())), dim3(kWideThreads), kWideLds, s, p, tilesM, tilesN);
    return hipGetLastError();
}

// The product's parts joined, and the column sums' along with them.
template <int FIN>
hipError_t launch_join(LinearParams p, bool wide, hipStream_t s)
{
    constexpr bool GLU = FIN == kFinFwdGlu;
    const int64_t cols = GLU ? p.N / 2 : p.N, tn = GLU ? kWide / 2 : kWide;
    const int64_t grid = wide ? p.cut.rest * (GLU ? 16 : 32) : (p.M * (cols / 8) + kThreads - 1) / kThreads;
    p.join_blocks = (int)(!wide && grid > 16384 ? 16384 : grid);
    const dim3 g((unsigned)(p.join_blocks + sums_join_blocks(p))), b(kThreads);
    if (wide)
        hipLaunchKernelGGL(linear_wide_join_kernel<FIN>, g, b, 0, s, p, (int)((p.M + kWide - 1) / kWide), (int)((cols + tn - 1) / tn));
    else
        hipLaunchKernelGGL(linear_join_kernel<FIN>, g, b, 0, s, p);
    return hipGetLastError();
}

template <bool ALA, bool ALB>
hipError_t launch_op(const LinearParams &p, int tile, hipStream_t s)
{
    switch (tile) {
    case kTile256: return launch_wide<ALA, ALB>(p, s);
    case kTile128: return launch_tile<ALA, ALB, 128, 128, 2, 2, 1, 2>(p, s);
    case kTile128Deep: return launch_tile<ALA, ALB, 128, 128, 2, 2, 1, 4>(p, s);
    case kTile64Deep: return launch_tile<ALA, ALB, 64, 128, 2, 2, 1, 6>(p, s);
    case kTile32Deep:
        if constexpr (ALA) return launch_tile<ALA, ALB, 32, 128, 1, 2, 1, 7>(p, s);
    default: return launch_tile<ALA, ALB, 64, 128, 2, 2, 1, 3>(p, s);
    }
}

hipError_t launch_few(const LinearParams &p, hipStream_t s)
{
    const bool glu = p.f.finish == kFinFwdGlu;
    const int64_t grid = ((glu ? p.N / 2 : p.N) + (glu ? 7 : 15)) / (glu ? 8 : 16);
    const dim3 g((unsigned)grid), b(kFewWaves * kWave);
    hipLaunchKernelGGL(linear_few_kernel, g, b, 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearParams &p0, int op, const LinearPlan &plan, hipStream_t s)
{
    LinearParams p = p0;
    p.splits = plan.splits;
    p.part = plan.part;
    p.cut = plan.cut;
    if (plan.tile == kTileFew) return launch_few(p, s);
    if (p.splits > 1) p.f.finish = kFinPartial;
    hipError_t e;
    if (plan.tile == kTileNarrow) e = launch_tile<true, true, 64, 32, 1, 1, 4, 6>(p, s);
    else if (op == kLinFwd) e = launch_op<true, true>(p, plan.tile, s);
    else if (op == kLinDgrad) e = launch_op<true, false>(p, plan.tile, s);
    else e = launch_op<false, false>(p, plan.tile, s);
    if (e != hipSuccess) return e;
    const bool wide = plan.tile == kTile256, join = wide ? p.cut.rest > 0 : p.splits > 1;
    if (p.sums.dbias) {
        // after the product, which leaves dy in the caches
        hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((p.sums.N + kColsumCols - 1) / kColsumCols), p.sums.parts), dim3(kThreads), 0,
                           s, p.sums);
        if (p.sums.parts > 1 && !join)
            hipLaunchKernelGGL(colsum_join_kernel, dim3((unsigned)sums_join_blocks(p)), dim3(kThreads), 0, s, p.sums);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!join) return hipSuccess;
    p.f.finish = p0.f.finish;
    switch (p.f.finish) {
    case kFinFwd: return launch_join<kFinFwd>(p, wide, s);
    case kFinFwdGlu: return launch_join<kFinFwdGlu>(p, wide, s);
    case kFinGrad: return launch_join<kFinGrad>(p, wide, s);
    default: return launch_join<kFinGradGlu>(p, wide, s);
    }
}

LinearPlan linear_plan(int op, int64_t M, int64_t N, int64_t K) { return plan_linear(op, M, N, K); }

int colsum_parts(int64_t M, int64_t N)
{
    const int64_t cols = (N + kColsumCols - 1) / kColsumCols;
    int64_t parts = (M + kColsumRows * 8 - 1) / (kColsumRows * 8);       // eight rows a thread at least
    const int64_t most = (1024 + cols - 1) / cols;
    if (parts > most) parts = most;
    return (int)(parts < 1 ? 1 : parts);
}

hipError_t launch_act_bwd(const uint16_t *dout, const uint16_t *c, uint16_t *dc, int64_t M, int64_t N, int act,
                          float limit, hipStream_t s)
{
    FinishParams f = {};
    f.out = dc;
    f.c = c;
    f.N = act == kActSwiglu ? N / 2 : N;
    f.ldo = N;
    f.finish = act == kActSwiglu ? kFinGradGlu : kFinGrad;
    f.act = act;
    f.limit = limit;
    const int64_t grid = (M * (f.N / 8) + kThreads - 1) / kThreads;
    const dim3 g((unsigned)(grid > 16384 ? 16384 : grid)), b(kThreads);
    if (act == kActSwiglu) hipLaunchKernelGGL(act_bwd_kernel<kFinGradGlu>, g, b, 0, s, dout, f, M);
    else hipLaunchKernelGGL(act_bwd_kernel<kFinGrad>, g, b, 0, s, dout, f, M);
    return hipGetLastError();
}

}  // namespace ptgg
