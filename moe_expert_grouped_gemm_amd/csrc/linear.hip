// linear.hip -- dense matrix product with bias, activation and residual in its
// epilogue, its data gradient (which ends in the activation's gradient) and its
// weight gradient.
//
//   forward  C[m, n] = sum_k x[m, k] w[n, k]      both operands along the reduction
//   dgrad    C[m, k] = sum_n dy[m, n] w[n, k]     w across it
//   wgrad    C[n, k] = sum_m dy[m, n] x[m, k]     both across it
//
// One kernel serves all three: a workgroup computes a TM x TN tile of C over
// one part of the reduction, in stages of 64 values through a ring of LDS
// slots filled by direct loads.  Operands keep in LDS the layout that they
// have in memory: along the reduction as rows of 128 bytes read with
// ds_read_b128, across it as 64 rows read with the transposing
// ds_read_b64_tr_b16.  Products are v_mfma_f32_32x32x16_bf16 with the operands
// swapped, so that a lane holds four neighbouring columns of one row and the
// tile passes through LDS in 16-byte pieces, still in fp32: bias, activation
// and residual are applied to unrounded sums and the result is rounded once.
// Where the tiles alone do not fill the chip the reduction is cut in parts
// whose fp32 sums a second kernel adds in order and finishes.
#include "dense.hpp"
#include "pipeline.hpp"
#include "rows.hpp"

namespace ptgg {

namespace {

template <int V>
struct IC { static constexpr int value = V; };

constexpr int kStage = 64;                    // reduction values of a stage

// ------------------------------------------------------------------ activations
// e^x to about an ulp: the product x log2(e) in two parts, its whole part by
// ldexp.  Past +-150 it is 0 or infinite (NaN becomes some number: the callers
// multiply by their argument).
__device__ __forceinline__ float exp_(float x)
{
    constexpr float kL = 1.44269502162933349609375f, kLow = 1.925963033500011e-8f;
    x = __builtin_amdgcn_fmed3f(x, -150.0f, 150.0f);
    const float n = __builtin_rintf(x * kL);
    const float f = __builtin_fmaf(x, kLow, __builtin_fmaf(x, kL, -n));
    return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}
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
__device__ __forceinline__ float glu_of(float g, float u, float lim)
{
    g = g > lim ? lim : g;
    u = u > lim ? lim : u < -lim ? -lim : u;
    return g * sigmoid_(g) * u;
}
__device__ __forceinline__ void glu_slope(float g0, float u0, float lim, float d, float &dg, float &du)
{
    const float g = g0 > lim ? lim : g0, u = u0 > lim ? lim : u0 < -lim ? -lim : u0;
    const float s = sigmoid_(g);
    dg = g0 > lim ? 0.0f : d * u * (s * (1.0f + g * (1.0f - s)));
    du = __builtin_fabsf(u0) > lim ? 0.0f : d * (g * s);
    if (g != g) du = dg;                 // a NaN gate makes both NaN, also where the sigmoid dropped it
}

// ------------------------------------------------------------------ finish
// Eight neighbouring sums v of row m and, for kFinFwdGlu, the eight ups u that
// belong to them; n: v's first column of the product.  Sums are fp32 until the
// one rounding of each output.
__device__ __forceinline__ void store8(const FinishParams &p, int64_t at, const float (&v)[8])
{
    if (p.f32) store_stream<true, false>(p.out, at, v);
    else store_stream<false, false>(p.out, at, v);
}

__device__ __forceinline__ void add_row8(const uint16_t *b, float (&v)[8])
{
    float f[8];
    unpack8(*(const uintx4 *)b, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += f[i];
}

__device__ __forceinline__ void add_residual8(const FinishParams &p, int64_t at, float (&v)[8])
{
    if (!p.residual) return;
    float f[8];
    if (p.f32) load_stream<true, false>(p.residual, at, f);
    else load_stream<false, false>(p.residual, at, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += f[i];
}

__device__ __forceinline__ void act8(float (&v)[8], int act)
{
    switch (act) {                       // one branch for the eight
#define PTGG_ACT(A)                                       \
    case A:                                               \
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
#define PTGG_ACT(A)                                       \
    case A:                                               \
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

__device__ __forceinline__ void finish8(const FinishParams &p, int64_t m, int64_t n, float (&v)[8], float (&u)[8])
{
    const int64_t at = m * p.ldo + n;
    if (p.finish == kFinFwd) {
        if (p.bias) add_row8(p.bias + n, v);
        if (p.save) *(uintx4 *)(p.save + m * p.N + n) = pack8(v);
        act8(v, p.act);
        add_residual8(p, at, v);
        store8(p, at, v);
    } else if (p.finish == kFinFwdGlu) {
        const int64_t I = p.N >> 1;
        if (p.bias) {
            add_row8(p.bias + n, v);
            add_row8(p.bias + I + n, u);
        }
        if (p.save) {
            *(uintx4 *)(p.save + m * p.N + n) = pack8(v);
            *(uintx4 *)(p.save + m * p.N + I + n) = pack8(u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = glu_of(v[i], u[i], p.limit);
        add_residual8(p, at, v);
        store8(p, at, v);
    } else if (p.finish == kFinGrad) {
        if (p.c) {
            float c[8];
            unpack8(*(const uintx4 *)(p.c + at), c);
            slope8(v, c, p.act);
        }
        add_residual8(p, at, v);
        store8(p, at, v);
    } else {
        const int64_t I = p.N;           // ldo is 2 N
        float g[8];
        unpack8(*(const uintx4 *)(p.c + at), g);
        unpack8(*(const uintx4 *)(p.c + at + I), u);
#pragma unroll
        for (int i = 0; i < 8; ++i) glu_slope(g[i], u[i], p.limit, v[i], g[i], u[i]);
        store8(p, at, g);
        store8(p, at + I, u);
    }
}

// ------------------------------------------------------------------ operands
__device__ __forceinline__ uint32_t clip_bytes(int64_t left) { return left <= 0 ? 0u : left > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)left; }

// Chunk swizzles of a stage in LDS.  Along the reduction (rows of 128 bytes):
// the 16 lanes of a ds_read_b128 pass, reading one chunk of 16 consecutive
// rows, cover all banks.  Across it (rows of CPR chunks): the four rows of a
// transposing read's 16 lanes fall on different banks.
__device__ __forceinline__ int along(int r, int c) { return c ^ ((r >> 1) & 7); }
template <int CPR>
__device__ __forceinline__ int across(int k, int c)
{
    return CPR >= 16 ? c ^ ((k & 3) << 2) : c ^ (((k >> 1) & 1) << 2);
}

// One operand of a tile: R rows (ALONG) or columns (!ALONG) of a stage, loaded
// by NT threads, 16 bytes each.  The base moves on by a stage with every
// issue, so that offsets stay small whatever the operand's size; loads at or
// past `left` bytes read zeros.  Along the reduction the two halves of the
// rows may lie apart (SwiGLU's gates and ups).
template <bool ALONG, int R, int NT>
struct Operand {
    static constexpr int NL = R * 128 / 16 / NT;
    static constexpr int CPR = ALONG ? 8 : R / 8;          // 16-byte chunks of an LDS row
    static constexpr int RPL = NT / CPR;                   // LDS rows per load
    static constexpr int HALVES = ALONG && NL >= 2 ? 2 : 1;
    static_assert(NL >= 1 && NT % CPR == 0 && RPL % 4 == 0, "loads of a stage");
    const uint8_t *base[HALVES];
    int64_t left[HALVES];
    int64_t step;
    uint32_t voff, rstep;
    int k;                                                 // this lane's first reduction value, ALONG

    // rows0, rows1: valid rows of the halves (ALONG); cols: valid columns (!ALONG)
    __device__ __forceinline__ void init(const uint16_t *p0, const uint16_t *p1, int rows0, int rows1, int64_t ld,
                                         int64_t klen, int64_t cols)
    {
        const int t = threadIdx.x, row = t / CPR;
        base[0] = (const uint8_t *)p0;
        rstep = (uint32_t)(RPL * ld * 2);
        if constexpr (ALONG) {
            const int chunk = along(row, t % CPR);
            left[0] = rows0 > 0 ? ((rows0 - 1) * ld + klen) * 2 : 0;
            voff = (uint32_t)(row * ld * 2) + chunk * 16;
            if constexpr (HALVES == 2) {
                base[1] = (const uint8_t *)p1;
                left[1] = rows1 > 0 ? ((rows1 - 1) * ld + klen) * 2 : 0;
            } else if (R == 32) {
                // one load takes both halves, which lie at most 32 rows apart
                const int64_t apart = (p1 - p0) * 2;
                if (rows1 > 0) left[0] = apart + ((rows1 - 1) * ld + klen) * 2;
                if (row >= R / 2) voff = (uint32_t)(apart + (row - R / 2) * ld * 2) + chunk * 16;
            }
            step = kStage * 2;
            k = chunk * 8;
        } else {
            const int chunk = across<CPR>(row, t % CPR);
            left[0] = klen > 0 ? ((klen - 1) * ld + cols) * 2 : 0;
            voff = (uint32_t)(row * ld * 2) + (uint32_t)min((int64_t)chunk * 8, cols - 8) * 2;
            step = kStage * ld * 2;
            k = 0;
        }
    }
    // Stage at reduction value k0 of klen into the slot at `lds`.
    __device__ __forceinline__ void issue(uint8_t *lds, int k0, int klen, int wave)
    {
        uint32_t v = voff;
        if (ALONG) v = k0 + k < klen ? voff : kOOB;
        uint8_t *d = lds + wave * kWave * 16;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int h = HALVES == 2 && i >= NL / 2;
            dma16(base[h], clip_bytes(left[h]), d + i * NT * 16, v, (uint32_t)(h ? i - NL / 2 : i) * rstep);
        }
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            base[h] += step;
            left[h] -= step;
        }
    }
};

template <int OFF>
__device__ __forceinline__ uintx2 read_tr(uint32_t addr)
{
    uintx2 v;
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
    return v;
}

// Fragments of NB blocks of 32 rows / columns at reduction step KS (16 values)
// of a stage.  at: per-lane address in the stage (frag_base), plus the slot.
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

template <bool ALONG, int R, int NB>
struct Frags {
    // across: one address per block, since the swizzle moves chunks of 32 bytes
    // among 64 columns
    static constexpr int NA = ALONG ? 1 : NB;
    uint32_t at[NA];
    __device__ __forceinline__ void init(uint32_t lds, int first)
    {
#pragma unroll
        for (int i = 0; i < NA; ++i) at[i] = lds + frag_base<ALONG, R>(first + 32 * i);
    }
    template <int KS>
    __device__ __forceinline__ void read(uint32_t slot, bf16x8 (&f)[NB], IC<KS>) const
    {
        if constexpr (ALONG) {
            read_along<0>((at[0] + slot) ^ (uint32_t)(KS << 5), f);
        } else {
            constexpr int O = KS * 16 * R * 2;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const uint32_t a = at[i] + slot;
                const uintx2 lo = read_tr<O>(a), hi = read_tr<O + 4 * R * 2>(a);
                f[i] = __builtin_bit_cast(bf16x8, uintx4{lo[0], lo[1], hi[0], hi[1]});
            }
        }
    }
    template <int I>
    __device__ __forceinline__ void read_along(uint32_t a, bf16x8 (&f)[NB]) const
    {
        if constexpr (I < NB) {
            f[I] = __builtin_bit_cast(bf16x8, ldsr_u128<I * 32 * 128>(a));
            read_along<I + 1>(a, f);
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
template <int NA, int NB>
__device__ __forceinline__ void pin_frags(bf16x8 (&a)[NA], bf16x8 (&b)[NB])
{
#pragma unroll
    for (int i = 0; i < NA; ++i) asm volatile("" : "+v"(a[i]));
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(b[i]));
}

// ------------------------------------------------------------------ kernel
// Tile TM x TN by WM x WN waves, times WK that share a stage's four steps of
// the reduction; NS slots of the ring.
template <int TM, int TN, int WM, int WN, int WK, int NS>
struct Shape {
    static constexpr int NT = kWave * WM * WN * WK;
    static constexpr int MI = TM / WM / 32, NJ = TN / WN / 32;
    static constexpr int SLOTA = TM * 128, SLOTB = TN * 128, SLOT = SLOTA + SLOTB, RING = NS * SLOT;
    static constexpr int PITCH = TN * 4 + 16;             // bytes of an fp32 row of the tile in LDS
    static constexpr int ER = TM * PITCH <= (96 << 10) ? TM : TM / 2;   // rows of the tile at a time
    static constexpr int LDS = RING > ER * PITCH ? RING : ER * PITCH;
    static constexpr int WGS = LDS * 2 <= (160 << 10) ? 2 : 1;    // workgroups on a CU
    static_assert(LDS <= (160 << 10) && ER % (TM / WM) == 0, "LDS of a tile");
};

// Logical workgroup number: consecutive ones share an XCD and its L2.
__device__ __forceinline__ uint32_t xcd_order()
{
    const uint32_t n = gridDim.x, b = blockIdx.x, q = n / 8, r = n % 8, x = b % 8;
    return x * q + min(x, r) + b / 8;
}

template <bool ALA, bool ALB, int TM, int TN, int WM, int WN, int WK, int NS>
__global__ __launch_bounds__(64 * WM * WN * WK, 2) void linear_kernel(LinearParams p, int tilesM, int tilesN)
{
    using S = Shape<TM, TN, WM, WN, WK, NS>;
    constexpr int NT = S::NT, MI = S::MI, NJ = S::NJ;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / WK / WN;

    const uint32_t id = xcd_order(), tiles = (uint32_t)tilesM * (uint32_t)tilesN;
    const int64_t split = id / tiles;
    int mt, nt;
    grouped_tile_order((int)(id % tiles), tilesM, tilesN, mt, nt);
    const int64_t m0 = (int64_t)mt * TM;
    const bool glu = p.f.finish == kFinFwdGlu;
    const int64_t kb = split * p.part;
    const int klen = (int)min(p.K - kb, p.part);
    // columns of the tile: n0 on, or with SwiGLU TN / 2 gates from n0 and the
    // same ups from N / 2 + n0
    const int64_t n0 = (int64_t)nt * (glu ? TN / 2 : TN);
    const int64_t half = p.N >> 1;

    Operand<ALA, TM, NT> oa;
    Operand<ALB, TN, NT> ob;
    {
        const int rows = (int)min(p.M - m0, (int64_t)TM);
        if (ALA) oa.init(p.a + m0 * p.lda + kb, p.a + (m0 + TM / 2) * p.lda + kb, rows, rows - TM / 2, p.lda, klen, 0);
        else oa.init(p.a + kb * p.lda + m0, nullptr, 0, 0, p.lda, klen, p.M - m0);
        if (ALB) {
            const int64_t n1 = glu ? half + n0 : n0 + TN / 2;
            const int rows0 = (int)min((glu ? half : p.N) - n0, (int64_t)(glu ? TN / 2 : TN));
            const int rows1 = glu ? rows0 : rows0 - TN / 2;
            ob.init(p.b + n0 * p.ldb + kb, p.b + n1 * p.ldb + kb, rows0, rows1, p.ldb, klen, 0);
        } else {
            ob.init(p.b + kb * p.ldb + n0, nullptr, 0, 0, p.ldb, klen, p.N - n0);
        }
    }
    const uint32_t lds0 = lds_addr(smem);
    Frags<ALA, TM, MI> ra;
    Frags<ALB, TN, NJ> rb;
    ra.init(lds0, wm * MI * 32);
    rb.init(lds0 + S::SLOTA, wn * NJ * 32);

    floatx16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    auto mma = [&](const bf16x8 (&af)[MI], const bf16x8 (&bf)[NJ]) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
    };

    constexpr int LOADSN = Operand<ALA, TM, NT>::NL + Operand<ALB, TN, NT>::NL;
    const int nk = (klen + kStage - 1) / kStage;
    auto issue = [&](int kt, int slot) {
        oa.issue(smem + slot * S::SLOT, kt * kStage, klen, wave);
        ob.issue(smem + slot * S::SLOT + S::SLOTA, kt * kStage, klen, wave);
    };
    // stages past the end load zeros, so that the waits need no cases
#pragma unroll
    for (int st = 0; st < NS - 1; ++st) issue(st, st);
    if constexpr (WK == 1) {
        bf16x8 fa[2][MI], fb[2][NJ];
        wait_vmcnt<(NS - 2) * LOADSN>();
        barrier();
        ra.read(0, fa[0], IC<0>{});
        rb.read(0, fb[0], IC<0>{});
        wait_frags(fa[0], fb[0]);
        int slot = 0;
        for (int kt = 0; kt < nk; ++kt) {
            const uint32_t so = (uint32_t)slot * S::SLOT;
            const int freed = slot == 0 ? NS - 1 : slot - 1, next = slot + 1 == NS ? 0 : slot + 1;
            issue(kt + NS - 1, freed);           // the slot that stage kt - 1 left at its closing barrier
            ra.read(so, fa[1], IC<1>{});
            rb.read(so, fb[1], IC<1>{});
            mma(fa[0], fb[0]);
            wait_frags(fa[1], fb[1]);
            ra.read(so, fa[0], IC<2>{});
            rb.read(so, fb[0], IC<2>{});
            mma(fa[1], fb[1]);
            wait_frags(fa[0], fb[0]);
            ra.read(so, fa[1], IC<3>{});
            rb.read(so, fb[1], IC<3>{});
            mma(fa[0], fb[0]);
            wait_frags(fa[1], fb[1]);
            wait_vmcnt<(NS - 2) * LOADSN>();     // stage kt + 1 has landed for this wave, and after the barrier for all
            barrier();
            const uint32_t sn = (uint32_t)next * S::SLOT;
            ra.read(sn, fa[0], IC<0>{});
            rb.read(sn, fb[0], IC<0>{});
            pin_frags(fa[1], fb[1]);
            mma(fa[1], fb[1]);
            wait_frags(fa[0], fb[0]);
            slot = next;
        }
    } else {
        static_assert(WK == 4, "a step of the stage per wave");
        bf16x8 fa[MI], fb[NJ];
        int slot = 0;
        for (int kt = 0; kt < nk; ++kt) {
            wait_vmcnt<(NS - 2) * LOADSN>();
            barrier();
            const uint32_t so = (uint32_t)slot * S::SLOT;
            switch (wk) {
            case 0: ra.read(so, fa, IC<0>{}); rb.read(so, fb, IC<0>{}); break;
            case 1: ra.read(so, fa, IC<1>{}); rb.read(so, fb, IC<1>{}); break;
            case 2: ra.read(so, fa, IC<2>{}); rb.read(so, fb, IC<2>{}); break;
            default: ra.read(so, fa, IC<3>{}); rb.read(so, fb, IC<3>{}); break;
            }
            wait_frags(fa, fb);
            issue(kt + NS - 1, slot == 0 ? NS - 1 : slot - 1);
            mma(fa, fb);
            slot = slot + 1 == NS ? 0 : slot + 1;
        }
    }
    wait_vmcnt<0>();                             // zeros of stages past the end may still be landing in the ring
    barrier();

    // ---- the tile through LDS in fp32: lane l holds of block (i, j) row l % 32
    // and columns (r / 4) 8 + (l / 32) 4 + r % 4
    const int64_t ncols = glu ? half : p.N;
#pragma unroll 1
    for (int e0 = 0; e0 < TM; e0 += S::ER) {
        const int row0 = wm * MI * 32 - e0;
        if (e0) __syncthreads();
#pragma unroll 1
        for (int w = 0; w < WK; ++w) {
            if (w) __syncthreads();
            if (WK > 1 && w != wk) continue;
            if (row0 < 0 || row0 >= S::ER) continue;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        floatx4 *d = (floatx4 *)(smem + (row0 + i * 32 + (lane & 31)) * S::PITCH +
                                                 (wn * NJ * 32 + j * 32 + q * 8 + (lane >> 5) * 4) * 4);
                        floatx4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                        *d = w ? *d + v : v;
                    }
        }
        __syncthreads();
        const int groups = glu ? TN / 16 : TN / 8;
        for (int i = threadIdx.x; i < S::ER * groups; i += NT) {
            const int r = i / groups, g = i - r * groups;
            const int64_t m = m0 + e0 + r, n = n0 + g * 8;
            if (m >= p.M || n >= ncols) continue;
            const uint8_t *src = smem + r * S::PITCH + g * 32;
            float v[8], u[8];
            *(floatx4 *)v = *(const floatx4 *)src;
            *(floatx4 *)(v + 4) = *(const floatx4 *)(src + 16);
            if (glu) {
                *(floatx4 *)u = *(const floatx4 *)(src + TN / 2 * 4);
                *(floatx4 *)(u + 4) = *(const floatx4 *)(src + TN / 2 * 4 + 16);
            }
            if (p.f.finish == kFinPartial) store_stream<true, false>(p.partials, (split * p.M + m) * p.N + n, v);
            else finish8(p.f, m, n, v, u);
        }
    }
}


// ------------------------------------------------------------------ few rows
// At most 64 rows against w [N, K]: w is read once, x comes from L2.  A
// workgroup takes 16 columns (8 gates and their ups), its eight waves the
// steps of 64 reduction values in turn: a wave's loads of a step are whole
// lines of 16 rows.  The reduction's values are taken in the order in which a
// lane's two 16-byte loads find them, alike for both operands.  The waves'
// sums meet in LDS and are added in order.
constexpr int kFewWaves = 8, kFewCols = 16;

template <int MT>
__global__ __launch_bounds__(kFewWaves * kWave) void linear_few_kernel(LinearParams p)
{
    constexpr int U = MT == 1 ? 4 : 2;                       // steps of a batch; two batches are in flight
    constexpr int PITCH = kFewCols + 4;
    __shared__ __attribute__((aligned(16))) float red[kFewWaves][MT * 16][PITCH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const bool glu = p.f.finish == kFinFwdGlu;
    const int64_t half = p.N >> 1;
    const int64_t n0 = (int64_t)blockIdx.x * (glu ? kFewCols / 2 : kFewCols);
    int64_t n = glu && r16 >= 8 ? half + n0 + r16 - 8 : n0 + r16;
    if (n >= p.N) n = p.N - 1;                               // read, never stored
    const uint16_t *w = p.b + n * p.ldb + q * 16;
    const uint16_t *x[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = p.a + min((int64_t)i * 16 + r16, p.M - 1) * p.lda + q * 16;
    floatx4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = floatx4{0, 0, 0, 0};

    struct Batch {
        uintx4 w[U][2], x[U][MT][2];
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
#pragma unroll
                for (int i = 0; i < MT; ++i) b.x[u][i][h] = *(const uintx4 *)(x[i] + s + h * 8);
            }
        }
    };
    auto mma = [&](const uintx4 &wv, const uintx4 &xv, int i) {
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv), __builtin_bit_cast(bf16x8, xv),
                                                         acc[i], 0, 0, 0);
    };
    auto use = [&](const Batch &b, int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u * kFewWaves >= full) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i) mma(b.w[u][h], b.x[u][i][h], i);
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
            uintx4 wv = *(const uintx4 *)(w + o);
            wv = ok ? wv : uintx4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uintx4 xv = *(const uintx4 *)(x[i] + o);
                xv = ok ? xv : uintx4{0, 0, 0, 0};
                mma(wv, xv, i);
            }
        }
    }
    // lane l: row l % 16 of x's block, columns (l / 16) 4 + r
#pragma unroll
    for (int i = 0; i < MT; ++i) *(floatx4 *)&red[wave][i * 16 + r16][q * 4] = acc[i];
    __syncthreads();
    const int groups = glu ? 1 : 2;
    for (int i = threadIdx.x; i < MT * 16 * groups; i += kFewWaves * kWave) {
        const int m = i / groups, g = i % groups;
        const int64_t nn = n0 + g * 8;
        if (m >= p.M || (!glu && nn >= p.N)) continue;
        float v[8] = {}, u[8] = {};
#pragma unroll
        for (int wv = 0; wv < kFewWaves; ++wv)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] += red[wv][m][g * 8 + j];
                if (glu) u[j] += red[wv][m][8 + j];
            }
        finish8(p.f, m, nn, v, u);
    }
}

// The parts' sums added in order, then what the tile itself would have done.
__global__ __launch_bounds__(kThreads) void linear_join_kernel(LinearParams p)
{
    const bool glu = p.f.finish == kFinFwdGlu;
    const int64_t half = p.N >> 1, groups = (glu ? half : p.N) / 8, total = p.M * groups;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t m = i / groups, n = (i - m * groups) * 8;
        float v[8] = {}, u[8] = {};
        for (int s = 0; s < p.splits; ++s) {
            float f[8];
            const int64_t at = (s * p.M + m) * p.N + n;
            load_stream<true, false>(p.partials, at, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += f[j];
            if (glu) {
                load_stream<true, false>(p.partials, at + half, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] += f[j];
            }
        }
        finish8(p.f, m, n, v, u);
    }
}

// ------------------------------------------------------------------ column sums
// A workgroup adds 64 columns over one part of the rows: 8 lanes of 8 columns,
// 32 rows side by side, joined in LDS in their order.
constexpr int kColsumCols = 64, kColsumRows = 32;
__global__ __launch_bounds__(kThreads) void colsum_kernel(const uint16_t *__restrict__ dy, float *dbias, float *partials,
                                                          int64_t M, int64_t N, int accumulate)
{
    __shared__ float s[kColsumRows][kColsumCols + 4];
    const int lane = threadIdx.x & 7, side = threadIdx.x >> 3;
    const int64_t n = (int64_t)blockIdx.x * kColsumCols + lane * 8;
    float v[8] = {};
    if (n < N) {
#pragma unroll 4
        for (int64_t r = (int64_t)blockIdx.y * kColsumRows + side; r < M; r += (int64_t)gridDim.y * kColsumRows) add_row8(dy + r * N + n, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[side][lane * 8 + j] = v[j];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * kColsumCols + threadIdx.x;
    if (threadIdx.x >= kColsumCols || c >= N) return;
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < kColsumRows; ++r) sum += s[r][threadIdx.x];
    if (gridDim.y > 1) partials[(int64_t)blockIdx.y * N + c] = sum;
    else dbias[c] = accumulate ? dbias[c] + sum : sum;
}

__global__ __launch_bounds__(kThreads) void colsum_join_kernel(const float *__restrict__ partials, float *dbias, int parts,
                                                               int64_t N, int accumulate)
{
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= N) return;
    float sum = 0.0f;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) sum += partials[(int64_t)i * N + c];
    dbias[c] = accumulate ? dbias[c] + sum : sum;
}

__global__ __launch_bounds__(kThreads) void act_bwd_kernel(const uint16_t *__restrict__ dout, FinishParams f, int64_t M)
{
    const int64_t groups = f.N / 8, total = M * groups;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t m = i / groups, n = (i - m * groups) * 8;
        float v[8], u[8];
        unpack8(*(const uintx4 *)(dout + m * f.N + n), v);
        finish8(f, m, n, v, u);
    }
}

// ------------------------------------------------------------------ plan and launch
enum Tile { kTileFew = 0, kTile256 = 1, kTile128 = 2, kTile64 = 3, kTileNarrow = 4 };
struct TileShape {
    int tm, tn, per_cu;      // workgroups of it that a CU holds
    float stage;             // us of a stage while a CU holds them
};
constexpr TileShape kTiles[] = {{64, 16, 1, 0}, {256, 256, 1, 1.3f}, {128, 128, 2, 1.0f}, {64, 128, 2, 0.8f}, {64, 32, 2, 0.5f}};

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
hipError_t launch_op(const LinearParams &p, int tile, hipStream_t s)
{
    switch (tile) {
    case kTile256: return launch_tile<ALA, ALB, 256, 256, 2, 4, 1, 2>(p, s);
    case kTile128: return launch_tile<ALA, ALB, 128, 128, 2, 2, 1, 2>(p, s);
    default: return launch_tile<ALA, ALB, 64, 128, 1, 4, 1, 3>(p, s);
    }
}

hipError_t launch_few(const LinearParams &p, hipStream_t s)
{
    const bool glu = p.f.finish == kFinFwdGlu;
    const int64_t grid = ((glu ? p.N / 2 : p.N) + (glu ? 7 : 15)) / (glu ? 8 : 16);
    const dim3 g((unsigned)grid), b(kFewWaves * kWave);
    if (p.M <= 16) hipLaunchKernelGGL(linear_few_kernel<1>, g, b, 0, s, p);
    else if (p.M <= 32) hipLaunchKernelGGL(linear_few_kernel<2>, g, b, 0, s, p);
    else hipLaunchKernelGGL(linear_few_kernel<4>, g, b, 0, s, p);
    return hipGetLastError();
}

}  // namespace

LinearPlan linear_plan(int op, int64_t M, int64_t N, int64_t K)
{
    LinearPlan best = {kTileFew, 1, (K + kStage - 1) / kStage * kStage, 0};
    if (op == kLinFwd && M <= 64) return best;
    const int64_t stages = (K + kStage - 1) / kStage;
    float cost = 0;
    for (int t = kTile256; t <= kTileNarrow; ++t) {
        const TileShape &sh = kTiles[t];
        if (t == kTileNarrow && (op != kLinFwd || N > 32)) continue;
        const int64_t tiles = ((M + sh.tm - 1) / sh.tm) * ((N + sh.tn - 1) / sh.tn);
        for (int want = 1; want <= 32 && (want == 1 || stages / want >= 4); want *= 2) {
            const int64_t per = stages > 0 ? (stages + want - 1) / want : 1, splits = stages > 0 ? (stages + per - 1) / per : 1;
            if (want > 1 && tiles * splits > 2048) break;
            const int64_t rounds = (tiles * splits + 256 * sh.per_cu - 1) / (256 * sh.per_cu);
            float c = (float)rounds * ((float)per * sh.stage + 3.0f);
            if (splits > 1) c += 3.0f + (float)(splits * M * N) * (8.0f / 4e6f);
            if (cost == 0 || c < cost) {
                cost = c;
                best = {t, (int)splits, per * kStage, splits > 1 ? splits * M * N * 4 : 0};
            }
        }
    }
    return best;
}

hipError_t launch_linear(const LinearParams &p0, int op, const LinearPlan &plan, hipStream_t s)
{
    LinearParams p = p0;
    p.splits = plan.splits;
    p.part = plan.part;
    if (plan.tile == kTileFew) return launch_few(p, s);
    if (p.splits > 1) p.f.finish = kFinPartial;
    hipError_t e;
    if (plan.tile == kTileNarrow) e = launch_tile<true, true, 64, 32, 1, 1, 4, 6>(p, s);
    else if (op == kLinFwd) e = launch_op<true, true>(p, plan.tile, s);
    else if (op == kLinDgrad) e = launch_op<true, false>(p, plan.tile, s);
    else e = launch_op<false, false>(p, plan.tile, s);
    if (e != hipSuccess || p.splits == 1) return e;
    p.f.finish = p0.f.finish;
    const int64_t items = p.M * ((p.f.finish == kFinFwdGlu ? p.N / 2 : p.N) / 8);
    const int64_t grid = (items + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)(grid > 16384 ? 16384 : grid)), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

int colsum_parts(int64_t M, int64_t N)
{
    const int64_t cols = (N + kColsumCols - 1) / kColsumCols;
    int64_t parts = (M + kColsumRows * 8 - 1) / (kColsumRows * 8);       // eight rows a thread at least
    const int64_t most = (1024 + cols - 1) / cols;
    if (parts > most) parts = most;
    return (int)(parts < 1 ? 1 : parts);
}

hipError_t launch_colsum(const uint16_t *dy, float *dbias, float *partials, int64_t M, int64_t N, int accumulate,
                         hipStream_t s)
{
    const int parts = colsum_parts(M, N);
    hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((N + kColsumCols - 1) / kColsumCols), parts), dim3(kThreads), 0, s, dy,
                       dbias, partials, M, N, accumulate);
    if (parts > 1)
        hipLaunchKernelGGL(colsum_join_kernel, dim3((unsigned)((N + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                           partials, dbias, parts, N, accumulate);
    return hipGetLastError();
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
    hipLaunchKernelGGL(act_bwd_kernel, dim3((unsigned)(grid > 16384 ? 16384 : grid)), dim3(kThreads), 0, s, dout, f, M);
    return hipGetLastError();
}

}  // namespace ptgg
