// few_tokens.hip -- the whole MoE layer for at most 64 tokens: router, FC1 +
// SwiGLU, FC2 and the weighted sum over each token's experts.
//
// The weights of the chosen experts are read once and everything else is
// small, so streaming them is the bound.  A wave owns 16 rows of one expert's
// matrix: the A operand of v_mfma_f32_16x16x32_bf16 (weights in 8 or 4 bits are
// widened in registers, exactly); the expert's tokens are the B operand, from
// LDS.  The order of the reduction is free, so a lane takes whichever
// consecutive elements its 16 bytes hold and reads the same ones of x.
//
// h = silu(gate) up is rounded to bf16 between the two products, as the grouped
// GEMM's SwiGLU epilogue does, so decoding and training see the same values.
#include "route_device.hpp"

namespace ptgg {

namespace {

constexpr int kFewThreads = 512;          // 8 waves share a block's tokens in LDS
constexpr int kWaves = kFewThreads / 64;
constexpr int kFewLds = 65536;            // token rows: two workgroups a CU
constexpr int kRows = 16;                 // weight rows of a tile
constexpr int kDepth = 4;                 // units of 2 KB that a wave keeps in flight
constexpr int kStage = 2;                 // 16-byte pieces of the token rows a thread has in flight

// Elements in 16 bytes of a row, and in a unit, the reduction's step: a whole
// 128-byte line of each of the tile's rows.
__host__ __device__ constexpr int piece_elems(int wt) { return wt == kFewBf16 ? 8 : wt == kFewMxfp8 ? 16 : 32; }
__host__ __device__ constexpr int unit_elems(int wt) { return 8 * piece_elems(wt); }
// LDS bytes of one token's row of K values: padded with zeros to whole units,
// and 16 bytes so that 16 rows start in different banks.
__host__ __device__ constexpr int x_pitch(int K, int wt)
{
    return (K + unit_elems(wt) - 1) / unit_elems(wt) * unit_elems(wt) * 2 + 16;
}
int row_cap(int K, int wt, int T)
{
    const int fit = kFewLds / x_pitch(K, wt), most = T < 16 ? T : 16;
    return fit < most ? fit : most;
}
// Waves that share a tile's reduction.  A wave has 8 KB of loads in flight and
// the card needs some 16 MB for its bandwidth, so the k experts of a single
// token should keep 2048 waves; a wave's share is a full ring at least.  The
// number of tokens does not enter: a token's sums do not depend on who shares
// its call.
int k_splits(int tiles, int k, int K, int wt)
{
    int s = 1;
    while (s < kWaves && (int64_t)tiles * k * s < 2048 && K / unit_elems(wt) >= 2 * s * kDepth) s *= 2;
    return s;
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// E8M0 byte as the scale operand of the conversions, which use its exponent
// alone (2^-127 for exponent 0); 255 is NaN.
__device__ __forceinline__ float e8m0(uint32_t e) { return bits_f32(e == 255u ? 0x7FC00000u : e << 23); }

// 16 bytes of 16 weight rows (lane % 16) times the tokens.  x: the same
// elements of token lane % 16; e: the scale byte.
template <int WT>
__device__ __forceinline__ void mma_piece(const uintx4 w, uint32_t e, const uint8_t *x, floatx4 (&acc)[2], int odd)
{
    if constexpr (WT == kFewBf16) {
        acc[odd] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), *(const bf16x8 *)x, acc[odd],
                                                           0, 0, 0);
    } else {
        const float f = e8m0(e);
#pragma unroll
        for (int i = 0; i < piece_elems(WT) / 8; ++i) {
            bf16x8 a;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf16x2_t v;
                if constexpr (WT == kFewMxfp8)
                    v = j & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + (j >> 1)], f, true)
                              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + (j >> 1)], f, false);
                else
                    v = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 0)
                        : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 1)
                        : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 3);
                a[2 * j] = v[0], a[2 * j + 1] = v[1];
            }
            acc[i & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, *(const bf16x8 *)(x + 16 * i), acc[i & 1], 0, 0, 0);
        }
    }
}

// One unit.  A load instruction takes a whole line of 8 rows, since half lines
// of 16 (what the matrix instruction's operand asks for) reach two thirds of
// the bandwidth: lo holds rows 0..7 and hi rows 8..15, lane l piece l / 8 of
// row l % 8.  Of the four lane groups g = l / 16, the lower eight lanes of lo
// hold piece 2 g and the upper eight piece 2 g + 1; swapping the upper half of
// lo with the lower half of hi gives the operands of pieces 2 g and 2 g + 1 of
// all 16 rows.
template <int WT>
__device__ __forceinline__ void mma_unit(const uintx4 lo, const uintx4 hi, uint32_t e, const uint8_t *x,
                                         floatx4 (&acc)[2])
{
    uintx4 p, q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // row_ror:8, written to lanes 8..15 of each 16 (bank mask 0xC) or 0..7
        p[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)lo[i], (int)hi[i], 0x128, 0xF, 0xC, false);
        q[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)hi[i], (int)lo[i], 0x128, 0xF, 0x3, false);
    }
    // a block of 32: one for both pieces (8 bits), or one each (4 bits, two bytes of e)
    mma_piece<WT>(p, e & 0xFFu, x, acc, 0);
    mma_piece<WT>(q, WT == kFewMxfp4 ? e >> 8 : e, x + 2 * piece_elems(WT), acc, 1);
}

// A wave's share of a tile: n units, and in the last split the rows' partial
// unit.  A ring of kDepth units (and their scale bytes) stays in flight; the
// scheduling barriers keep each reload right behind the product that frees its
// registers.  Every load of start() is unconditional and inside its row, so
// that the wait for the token rows, issued before, leaves them in flight.
template <int WT>
struct Stream {
    static constexpr int EB = WT == kFewMxfp8 ? 4 : 8;              // scale bytes of a row per unit
    static constexpr int EL = WT == kFewMxfp8 ? 1 : 2;              // and of a lane
    static constexpr int XB = unit_elems(WT) * 2;                   // bytes of a token per unit
    const uint8_t *w0, *w1, *s;
    int n;
    uintx4 lo[kDepth], hi[kDepth], last_lo, last_hi;
    uint32_t e[kDepth], last_e;

    static __device__ __forceinline__ uint32_t scale_at(const uint8_t *p)
    {
        if constexpr (EL == 1) return *p;
        uint16_t v;
        __builtin_memcpy(&v, p, 2);                                 // rows of K/32 bytes start anywhere
        return v;
    }
    __device__ __forceinline__ void load(int i, int unit)
    {
        if constexpr (WT != kFewBf16) {
            e[i] = scale_at(s + unit * EB);
            __builtin_amdgcn_sched_barrier(0);
        }
        lo[i] = __builtin_nontemporal_load((const uintx4 *)(w0 + unit * 128));
        __builtin_amdgcn_sched_barrier(0);
        hi[i] = __builtin_nontemporal_load((const uintx4 *)(w1 + unit * 128));
        __builtin_amdgcn_sched_barrier(0);
    }
    // row0: the weight row of lane % 8, row1 = that of lane % 8 + 8; scales:
    // those of the row of lane % 16, any: the tensor of them
    __device__ __forceinline__ void start(const uint8_t *row0, const uint8_t *row1, const uint8_t *scales,
                                          const uint8_t *any, int K, int split, int splits)
    {
        const int lane = threadIdx.x & 63, piece = lane >> 3, g = lane >> 4;
        const int full = K / unit_elems(WT), rem = K % unit_elems(WT);
        const int bytes = K * 16 / piece_elems(WT);
        const int first = full * split / splits;
        n = full * (split + 1) / splits - first;
        // a row shorter than a unit has no full one: any of its bytes will do
        const int at = first * 128 + min(piece * 16, bytes - 16);
        w0 = row0 + at;
        w1 = row1 + at;
        s = full ? scales + first * EB + g * EL : any;
        const int tail = min(full * 128 + piece * 16, bytes - 16);
        const bool has = split == splits - 1 && piece * piece_elems(WT) < rem;
        last_lo = *(const uintx4 *)(row0 + tail);
        last_hi = *(const uintx4 *)(row1 + tail);
        last_e = 0;
        if constexpr (WT != kFewBf16) {
            const int b = full * EB + g * EL, end = K / 32 - 1;
            last_e = scales[min(b, end)];
            if (EL == 2) last_e |= (uint32_t)scales[min(b + 1, end)] << 8;
        }
        __builtin_amdgcn_sched_barrier(0);
        // in the ring's order, so that the first turn's waits are those of the others
#pragma unroll
        for (int i = 0; i < kDepth; ++i) load(i, max(min(i, n - 1), 0));
        // pieces past the rows' end are zeros (x is zero there too, and their scales are some block's of
        // the row), and so is the whole unit for the earlier splits
        if (!has) last_lo = last_hi = uintx4{0, 0, 0, 0};
    }
    // x: LDS row of token lane % 16, from the lane group's elements of the
    // split's first unit; x_last: from those of the partial unit.  Returns rows
    // 4 (lane / 16) + 0..3 of token lane % 16.
    __device__ __forceinline__ floatx4 product(const uint8_t *x, const uint8_t *x_last, bool tail)
    {
        floatx4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (; n >= 2 * kDepth; n -= kDepth) {
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                mma_unit<WT>(lo[i], hi[i], e[i], x + i * XB, acc);
                load(i, kDepth + i);
            }
            w0 += kDepth * 128, w1 += kDepth * 128, s += kDepth * EB, x += kDepth * XB;
        }
        if (n >= kDepth) {
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                mma_unit<WT>(lo[i], hi[i], e[i], x + i * XB, acc);
                if (kDepth + i < n) load(i, kDepth + i);
            }
            n -= kDepth, x += kDepth * XB;
        }
#pragma unroll
        for (int i = 0; i < kDepth - 1; ++i)
            if (i < n) mma_unit<WT>(lo[i], hi[i], e[i], x + i * XB, acc);
        if (tail) mma_unit<WT>(last_lo, last_hi, last_e, x_last, acc);
        return acc[0] + acc[1];
    }
};

// A block's token rows into LDS, zeros to the end of the last unit: batches of
// kStage pieces a thread, the last of them issued before and written after the
// weights' stream is started.
struct Stage {
    uintx4 v[kStage];
    int at;
    template <class Row>
    __device__ __forceinline__ void load(int pieces, int all, int K, Row row)
    {
#pragma unroll
        for (int q = 0; q < kStage; ++q) {
            const int i = min(at + q * kFewThreads + (int)threadIdx.x, all - 1);
            const int r = i / pieces, c = i - r * pieces;
            v[q] = *(const uintx4 *)(row(r) + min(c * 8, K - 8));
            if (c * 8 >= K) v[q] = uintx4{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ void store(uint8_t *lds, int pitch, int pieces, int all) const
    {
#pragma unroll
        for (int q = 0; q < kStage; ++q) {
            // past the end: into row 0's padding, which nothing reads (a branch would pull the load behind it)
            const int i = at + q * kFewThreads + (int)threadIdx.x;
            *(uintx4 *)(lds + (i < all ? i / pieces * pitch + i % pieces * 16 : pitch - 16)) = v[q];
        }
    }
    template <class Row>
    __device__ __forceinline__ void issue(uint8_t *lds, int pitch, int m, int K, Row row)
    {
        const int pieces = (pitch - 16) / 16, all = m * pieces;
        for (at = 0; at + kStage * kFewThreads < all; at += kStage * kFewThreads) {
            load(pieces, all, K, row);
            store(lds, pitch, pieces, all);
        }
        load(pieces, all, K, row);
    }
    __device__ __forceinline__ void finish(uint8_t *lds, int pitch, int m) const
    {
        const int pieces = (pitch - 16) / 16;
        store(lds, pitch, pieces, m * pieces);
    }
};

// The partial sums of a tile's splits, added in their order by the first.
__device__ __forceinline__ floatx4 join_splits(uint8_t *lds, floatx4 c, int split, int splits)
{
    floatx4 *part = (floatx4 *)lds + threadIdx.x;
    if (splits > 1) {
        if (split) *part = c;
        __syncthreads();
        if (!split)
            for (int i = 1; i < splits; ++i) c += part[i * 64];
    }
    return c;
}

__host__ __device__ constexpr int row_bytes(int K, int wt) { return wt == kFewBf16 ? K * 2 : wt == kFewMxfp8 ? K : K / 2; }

// The product of a tile that both kernels share.  load_row, step: the weight
// row (counted over all experts) that this lane loads, and from there to its
// second; row: the one whose products it takes part in; token_row: the block's
// rows of x or h.
template <int WT, class Row>
__device__ __forceinline__ floatx4 block_product(uint8_t *lds, const uint8_t *w, const uint8_t *scales, int64_t load_row,
                                                 int step, int64_t row, int m, int K, int split, int splits,
                                                 Row token_row)
{
    const int pitch = x_pitch(K, WT), lane = threadIdx.x & 63, g = lane >> 4;
    const uint8_t *row0 = w + load_row * row_bytes(K, WT);
    Stage st;
    Stream<WT> ws;
    st.issue(lds, pitch, m, K, token_row);
    ws.start(row0, row0 + (int64_t)step * row_bytes(K, WT), scales + row * (K / 32), scales, K,
             split, splits);
    st.finish(lds, pitch, m);
    __syncthreads();
    constexpr int XB = unit_elems(WT) * 2;
    const int full = K / unit_elems(WT);
    const uint8_t *x = lds + min(lane & 15, m - 1) * pitch + g * piece_elems(WT) * 4;
    const floatx4 c = ws.product(x + full * split / splits * XB, x + full * XB,
                                 K % unit_elems(WT) != 0 && split == splits - 1);
    if (splits > 1) __syncthreads();          // the token rows make room for the partial sums
    return join_splits(lds, c, split, splits);
}

// FC1 and SwiGLU: a tile is 8 gate rows and the 8 up rows of the same inner
// values, ordered so that a lane gets two gates and their two ups.
template <int WT>
__global__ __launch_bounds__(kFewThreads, 4) void few_fc1_kernel(FewParams p, int splits)
{
    extern __shared__ __align__(16) uint8_t lds[];
    const FewBlock *blk = (const FewBlock *)(p.plan + 4) + blockIdx.y;
    const int blocks = p.plan[0], e = blk->expert, row0 = blk->row0, m = blk->rows;
    const uintx4 tokens = *(const uintx4 *)blk->token;
    if ((int)blockIdx.y >= blocks) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int id = (int)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int split = id % splits, j0 = id / splits * 8;
    // waves past the last tile repeat it and store nothing
    const int64_t tile = (int64_t)e * 2 * p.I + min(j0, p.I - 8);
    const auto row = [&](int i) { return tile + ((i & 2) ? p.I : 0) + (i >> 2) * 2 + (i & 1); };
    const floatx4 c = block_product<WT>(lds, p.w1, p.w1s, row(lane & 7), 4, row(r), m, p.H, split, splits, [&](int i) {
        return p.x + (int64_t)((tokens[i >> 2] >> (8 * (i & 3))) & 0xFFu) * p.H;
    });
    if (j0 < p.I && !split && r < m)
        *(bf16x2_t *)(p.h + (int64_t)(row0 + r) * p.I + j0 + 2 * g) =
            bf16x2_t{(__bf16)silu_mul(c[0], c[2], p.swiglu_limit), (__bf16)silu_mul(c[1], c[3], p.swiglu_limit)};
}

template <int WT>
__global__ __launch_bounds__(kFewThreads, 4) void few_fc2_kernel(FewParams p, int splits)
{
    extern __shared__ __align__(16) uint8_t lds[];
    const FewBlock *blk = (const FewBlock *)(p.plan + 4) + blockIdx.y;
    const int blocks = p.plan[0], e = blk->expert, row0 = blk->row0, m = blk->rows;
    if ((int)blockIdx.y >= blocks) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int id = (int)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int split = id % splits, n0 = id / splits * kRows;
    // H % 16 may be 8: the rows past the end repeat the tile's first eight
    const int64_t tile = (int64_t)e * p.H + min(n0, p.H - 8);
    const int step = n0 + 8 < p.H ? 8 : 0;
    const floatx4 c = block_product<WT>(lds, p.w2, p.w2s, tile + (lane & 7), step, tile + (lane & 7) + (r >> 3) * step, m,
                                        p.I, split, splits, [&](int i) { return p.h + (int64_t)(row0 + i) * p.I; });
    if (!split && r < m && n0 + 4 * g < p.H) *(floatx4 *)(p.y + (int64_t)(row0 + r) * p.H + n0 + 4 * g) = c;
}

// out[t] = sum over the slots, in their order, of weight times the expert's row.
__global__ __launch_bounds__(kThreads) void few_sum_kernel(FewParams p)
{
    const int t = blockIdx.y, c = ((int)blockIdx.x * kThreads + (int)threadIdx.x) * 4;
    if (c >= p.H) return;
    floatx4 sum = {0, 0, 0, 0};
    // four slots' loads at a time
    for (int j0 = 0; j0 < p.k; j0 += 4) {
        int row[4];
        float w[4];
        floatx4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = t * p.k + min(j0 + j, p.k - 1);
            row[j] = j0 + j < p.k ? p.route.row_of[at] : -1;
            w[j] = p.route.topk_weights[at];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (row[j] >= 0) v[j] = *(const floatx4 *)(p.y + (int64_t)row[j] * p.H + c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (row[j] >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(w[j], v[j][i], sum[i]);
            }
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
    const int t1 = p.I / 8, t2 = (p.H + kRows - 1) / kRows;
    const int s1 = k_splits(t1, p.k, p.H, WT), s2 = k_splits(t2, p.k, p.I, WT);
    const int l1 = cap * x_pitch(p.H, WT), l2 = cap * x_pitch(p.I, WT), room = kFewThreads * 16;
    hipLaunchKernelGGL(few_fc1_kernel<WT>, dim3((unsigned)((t1 * s1 + kWaves - 1) / kWaves), (unsigned)blocks),
                       dim3(kFewThreads), l1 > room ? l1 : room, s, p, s1);
    hipLaunchKernelGGL(few_fc2_kernel<WT>, dim3((unsigned)((t2 * s2 + kWaves - 1) / kWaves), (unsigned)blocks),
                       dim3(kFewThreads), l2 > room ? l2 : room, s, p, s2);
    hipLaunchKernelGGL(few_sum_kernel, dim3((unsigned)((p.H / 4 + kThreads - 1) / kThreads), (unsigned)p.T),
                       dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace

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
