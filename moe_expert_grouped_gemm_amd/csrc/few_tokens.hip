// few_tokens.hip -- the whole MoE layer for at most 64 tokens: router, FC1 +
// SwiGLU, FC2 and the weighted sum over each token's experts.
//
// The weights of the chosen experts are read once and everything else is
// small, so streaming them is the bound.  A wave owns 16 rows of one expert's
// matrix: the A operand of v_mfma_f32_16x16x32_bf16; the expert's tokens are the
// B operand, from LDS.  The order of the reduction is free, so a lane takes
// whichever consecutive elements its 16 bytes hold and reads the same ones of x.
// Weights in 8 or 4 bits are widened in registers, exactly where bf16 holds a
// value of that size: below 2^-126 in its steps of 2^-133, above 3.39e38 as
// infinite.
//
// h = silu(gate) up is rounded to bf16 between the two products, as the grouped
// GEMM's SwiGLU epilogue does, so decoding and training see the same values.
#include <type_traits>

#include "route_device.hpp"

namespace ptgg {

namespace {

constexpr int kCuWaves = 16;              // that a CU holds of these kernels, in 4, 2 or 1 workgroups of 4, 8 or 16
constexpr int kCuLds = 160 * 1024;
constexpr int kRows = 16;                 // weight rows of a tile
constexpr int kDepth = 4;                 // units of 2 KB that a wave keeps in flight
constexpr int kScalePieces = 3;           // 8-byte pieces of scales a thread moves
constexpr int kTurns = 4;                 // places of a row where tiles start that would meet in memory's channels

// Elements in 16 bytes of a row, and in a unit, the reduction's step: a whole
// 128-byte line of each of the tile's rows.
__host__ __device__ constexpr int piece_elems(int wt) { return wt == kFewBf16 ? 8 : wt == kFewMxfp8 ? 16 : 32; }
__host__ __device__ constexpr int unit_elems(int wt) { return 8 * piece_elems(wt); }
__host__ __device__ constexpr int units_of(int K, int wt) { return (K + unit_elems(wt) - 1) / unit_elems(wt); }
__host__ __device__ constexpr int row_bytes(int K, int wt) { return K / piece_elems(wt) * 16; }
// LDS bytes of one token's row of K values: padded with zeros to whole units,
// and 16 bytes so that 16 rows start in different banks.
__host__ __device__ constexpr int x_pitch(int K, int wt) { return units_of(K, wt) * unit_elems(wt) * 2 + 16; }
// Scales of a workgroup's waves / splits tiles.
__host__ __device__ constexpr int scale_region(int K, int wt, int waves, int splits)
{
    return wt == kFewBf16 ? 0 : waves / splits * kRows * (K / 32);
}

// How a product is laid over the waves: `splits` waves share a tile's
// reduction, a workgroup does waves / splits tiles (a group).  A wave's stream
// should hold some 16 KB -- twice its ring; longer ones leave too few workgroups
// to share out evenly, shorter ones are all start and end.  The k experts of a
// single token should still keep 512 waves while that leaves a stream 8 KB, and
// 256 in any case.  Measured, FC1 / FC2 in us with 1, 2, 4, 8 waves to a tile:
// 1 token, 4 experts of 2880 x 2880 bf16 (92 KB tiles): 24.8 / 22.8, 26.8 / 14.4,
// 22.4 / 15.2, 22.5 / 13.2; 7 tokens, 4096 x 2048 MXFP4 (32 and 16 KB): 49 / 27,
// 47 / 31, 58 / 48, 95 / 88; 64 tokens, the same in bf16 (131 and 65 KB): 551 / 307,
// 570 / 281, 558 / 291, 604 / 320 (there the rule's 4 and 4 are 1 and 4% from the
// best).  The layer, where 256 or 512 waves are asked for whatever the stream: 24
// tokens on 2 of 60 MXFP4 experts of 2016 x 1504 (16 and 12 KB) 43.2 and 46.3, 16 on 3
// of 8 MXFP8 of 1056 x 800 (17 and 13 KB) 20.6 and 19.7.
// The number of tokens does not enter, here or in where a stream starts (Path): a
// token's sums do not depend on who shares its call.
struct Layout {
    int tiles, splits, groups, lds_fixed;
};
Layout layout_of(int tiles, int k, int K, int wt, int waves)
{
    int s = 1;
    const int bytes = kRows * row_bytes(K, wt);
    const auto scales = [&] { return scale_region(K, wt, kCuWaves, s); };   // of workgroups that fill a CU
    const auto short_of_waves = [&] { return (int64_t)tiles * k * s < (bytes / (2 * s) >= 8 * 1024 ? 512 : 256); };
    while (units_of(K, wt) >= 2 * s &&
           (scales() > kCuWaves * 64 * 8 * kScalePieces ||
            (s < 4 && (bytes / (2 * s) >= 15 * 1024 || short_of_waves()))))
        s *= 2;
    const int fixed = scale_region(K, wt, waves, s) + (s > 1 ? waves * 64 * 16 : 0);   // and the partial sums
    return {tiles, s, (tiles * s + waves - 1) / waves, fixed};
}
// Rows a block may have for `per_cu` of a product's workgroups to fit a CU.
int row_cap(const Layout &l, int K, int wt, int T, int per_cu)
{
    const int fit = (kCuLds / per_cu - l.lds_fixed) / x_pitch(K, wt), most = T < 16 ? T : 16;
    return fit < most ? fit : most;
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

// A block's token rows into LDS, zeros to the end of the last unit: batches of
// kStage pieces a thread, the last of them issued before and written after the
// weights' stream is started.
template <int THREADS>
struct Stage {
    // 16-byte pieces a thread has in flight: the large workgroups hold many rows (64 tokens, 8 experts of 4032 x 1984
    // bf16: 196 us with 2, 188 with 4), the small ones few (12 tokens, 60 of 736 x 608 8 bits: 24.4 and 25.2)
    static constexpr int kStage = THREADS == 64 * kCuWaves ? 4 : 2;
    uintx4 v[kStage];
    int at;
    template <class Row>
    __device__ __forceinline__ void load(int pieces, int all, int K, Row row)
    {
#pragma unroll
        for (int q = 0; q < kStage; ++q) {
            const int i = min(at + q * THREADS + (int)threadIdx.x, all - 1);
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
            const int i = at + q * THREADS + (int)threadIdx.x;
            *(uintx4 *)(lds + (i < all ? i / pieces * pitch + i % pieces * 16 : pitch - 16)) = v[q];
        }
    }
    template <class Row>
    __device__ __forceinline__ void issue(uint8_t *lds, int pitch, int m, int K, Row row)
    {
        const int pieces = (pitch - 16) / 16, all = m * pieces;
        for (at = 0; at + kStage * THREADS < all; at += kStage * THREADS) {
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

// One expert's matrix as a product's tiles see it.  FC1: a tile is 8 gate rows
// and the 8 up rows of the same inner values, ordered so that a lane's four
// sums are two gates and their two ups.  FC2: 16 rows in a row.
template <int PHASE>
struct Rows {
    int rows, inner;                      // of the matrix; gate rows (FC1)
    // Row of index i < 16 in a tile, from the tile's first, and where it lies
    // among the scales of a group of `tiles` (the gates', then the ups').
    __device__ __forceinline__ int row(int i) const
    {
        return PHASE == 1 ? ((i & 2) ? inner : 0) + (i >> 2) * 2 + (i & 1) : i;
    }
    __device__ __forceinline__ int scale_row(int slot, int i, int tiles) const
    {
        return PHASE == 1 ? ((i & 2) ? tiles * 8 : 0) + slot * 8 + (i >> 2) * 2 + (i & 1) : slot * kRows + i;
    }
    static constexpr int step = PHASE == 1 ? 8 : kRows;   // rows from tile to tile
    static constexpr int half = PHASE == 1 ? 4 : 8;       // from row(i) to row(i + 8)
};

// How the rows lie.  kShared: lines hold the end of one row and the start of
// the next, or two units' halves, and the second reader must find them in the
// caches (2880-byte rows: 87.7 us cached, 94.1 not; 2048-byte rows: 51.6 and
// 48.5).  kLines: whole lines, each of them read once.  kTurned: also a multiple
// of 4096 bytes apart, so that waves at the same unit of their rows would meet
// in a few of the memory's channels: consecutive tiles start at kTurns places of
// their rows and go round (8192-byte rows: 614 -> 548 us; the turn costs the
// others 1%).  The place follows from the tile's number alone, not from the tiles
// of a workgroup, whose waves follow from the number of tokens: a token's sums
// keep their order.  With 2, 4, 8 and 16 places: 178.4, 177.8, 178.4, 179.1 us
// (geometric mean of 12 layers of 1 to 64 tokens).
enum Path { kShared = 0, kLines = 1, kTurned = 2 };

// The products of one block with a group of tiles, one to `splits` waves.  A
// wave's stream of units is a ring of kDepth of them in flight; the scheduling
// barriers keep each reload right behind the product that frees its registers.
// It starts between the loads of the token rows and the wait for them.  The
// scales of the group lie in LDS: rows of K/32 bytes read a few at a time would
// ask for as many lines as the weights do.  store(tile, c): rows
// 4 (lane / 16) + 0..3 of token lane % 16.
template <int WT, int PHASE, int PATH, int WAVES, class Row, class Store>
__device__ __forceinline__ void block_product(uint8_t *lds, const uint8_t *w, const uint8_t *scales, Rows<PHASE> geo,
                                              const Layout &l, int m, int K, int group, Row token_row, Store store)
{
    constexpr int EB = WT == kFewMxfp8 ? 4 : 8, EL = WT == kFewMxfp8 ? 1 : 2;   // scale bytes of a unit, of a lane
    constexpr int XB = unit_elems(WT) * 2, THREADS = 64 * WAVES;
    constexpr bool MX = WT != kFewBf16, NT = PATH != kShared;
    const int pitch = x_pitch(K, WT), rb = row_bytes(K, WT), sb = K / 32, units = units_of(K, WT);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, piece = lane >> 3;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int splits = l.splits, tiles = WAVES / splits, split = wave % splits, slot = wave / splits;
    const int first = units * split / splits;
    const int tile = group * tiles + slot, n = units * (split + 1) / splits - first;
    const int start = PATH == kTurned ? n * (tile % kTurns) / kTurns : 0;
    uint8_t *s_part = lds, *s_scale = lds + (splits > 1 ? THREADS * 16 : 0);
    const int region = MX ? tiles * kRows * sb : 0;
    uint8_t *s_x = s_scale + region;

    Stage<THREADS> st;
    st.issue(s_x, pitch, m, K, token_row);
    // the group's scales, 8 bytes a piece (its rows are whole pieces); past the matrix: its last ones
    uintx2 sv[kScalePieces];
    if constexpr (MX) {
        const int run = PHASE == 1 ? region / 2 : region;              // bytes of consecutive rows
        const int end = (PHASE == 1 ? geo.inner : geo.rows) * sb;
#pragma unroll
        for (int i = 0; i < kScalePieces; ++i) {
            int at = (i * THREADS + (int)threadIdx.x) * 8, from = 0;
            if (PHASE == 1 && at >= run) at -= run, from = end;
            __builtin_memcpy(&sv[i], scales + from + min(group * run + at, end - 8), 8);
        }
    }

    // the stream: a scalar address and the lanes' offsets from it; past the last tile: that one again.  The last
    // tile of FC2 may have 8 rows only: those twice.
    const int t = min(tile, l.tiles - 1);
    const uint8_t *wp = w + (int64_t)t * geo.step * rb + first * 128;
    const uint32_t off = (uint32_t)geo.row(lane & 7) * rb + piece * 16;
    const uint32_t off_hi = off + (uint32_t)((PHASE == 2 && t * kRows + 8 >= geo.rows) ? 0 : geo.half * rb);
    // the last unit may be short: its pieces past the end read the row's last one and count as zeros (the token
    // rows are zero there too)
    const int short_by = units * 128 - rb;
    const bool cut = short_by != 0 && split == splits - 1;
    const uint32_t back = (uint32_t)max(piece * 16 - (128 - short_by - 16), 0);
    uintx4 lo[kDepth], hi[kDepth];
    int done = 0;                                                      // units behind wp, x and ep
    const auto unit_at = [&](int i) {                                  // the i-th from there, counted from them
        if (PATH != kTurned) return i;
        const int u = start + done + i;
        return u >= n ? u - n : u;
    };
    const auto load = [&](int i, int unit, bool fill = false) {
        const int u = unit_at(unit);
        const uint32_t b = cut && u == n - 1 - (PATH == kTurned ? 0 : done) ? back : 0;
        const uintx4 *p = (const uintx4 *)(wp + u * 128 + (off - b)), *q = (const uintx4 *)(wp + u * 128 + (off_hi - b));
        // what a short stream leaves of the ring: one piece for all lanes, which nothing uses (a branch would make the
        // waits below count on fewer loads)
        if (fill && unit >= n) p = q = (const uintx4 *)w;
        lo[i] = NT ? __builtin_nontemporal_load(p) : *p;
        __builtin_amdgcn_sched_barrier(0);
        hi[i] = NT ? __builtin_nontemporal_load(q) : *q;
        __builtin_amdgcn_sched_barrier(0);
    };
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kDepth; ++i) load(i, i, true);

    st.finish(s_x, pitch, m);
    if constexpr (MX) {
#pragma unroll
        for (int i = 0; i < kScalePieces; ++i) {
            const int at = (i * THREADS + (int)threadIdx.x) * 8;
            if (at < region) *(uintx2 *)(s_scale + at) = sv[i];
        }
    }
    __syncthreads();

    const uint8_t *x = s_x + min(r, m - 1) * pitch + g * piece_elems(WT) * 4 + first * XB;
    const uint8_t *ep = s_scale + geo.scale_row(slot, r, tiles) * sb + first * EB + g * EL;
    floatx4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    const auto scale = [&](int unit) -> uint32_t {
        if constexpr (!MX) return 0;
        if (EL == 1) return ep[unit * EB];
        uint16_t v;                                                    // rows of K/32 bytes start anywhere
        __builtin_memcpy(&v, ep + unit * EB, 2);
        return v;
    };
    const auto multiply = [&](int i, int unit) {
        const int u = unit_at(unit);
        uint32_t e = scale(u);
        if (cut && u == n - 1 - (PATH == kTurned ? 0 : done)) {
            if (piece * 16 >= 128 - short_by) lo[i] = hi[i] = uintx4{0, 0, 0, 0};
            // scales past the row's end are another's or none: zeros times a NaN would not be zeros
            if constexpr (MX) {
                const int b = (units - 1) * EB + g * EL;
                if (b >= sb) e = 0;
                if (EL == 2 && b + 1 >= sb) e &= 0xFFu;
            }
        }
        mma_unit<WT>(lo[i], hi[i], e, x + u * XB, acc);
    };
    const auto advance = [&] {
        done += kDepth;
        if (PATH != kTurned) wp += kDepth * 128, x += kDepth * XB, ep += kDepth * EB;
    };
    for (; n - done >= 2 * kDepth; advance()) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            multiply(i, i);
            load(i, kDepth + i);
        }
    }
    if (n - done >= kDepth) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            multiply(i, i);
            if (done + kDepth + i < n) load(i, kDepth + i);
        }
        advance();
    }
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i)
        if (done + i < n) multiply(i, i);

    floatx4 c = acc[0] + acc[1];
    if (splits > 1) {
        floatx4 *part = (floatx4 *)s_part + threadIdx.x;
        if (split) *part = c;
        __syncthreads();
        if (!split)
            for (int j = 1; j < splits; ++j) c += part[j * 64];
    }
    if (!split && tile < l.tiles && r < m) store(tile, c);
}

// Waves of a SIMD that the registers have to leave room for.  Short rows' LDS lets a third workgroup of 8 waves into a
// CU, for which 8-bit weights need 80 registers instead of 84 (12 tokens, 60 experts, 736 x 608: 26.8 us to 25.2).
constexpr int waves_per_simd(int wt, int waves) { return wt == kFewMxfp8 && waves <= 8 ? 6 : 4; }

// Which block and group of tiles a workgroup takes.  An expert's blocks read
// the same weights: eight groups of them at a time, so that a group's blocks
// start together and on one XCD (workgroups go round the eight), whose L2 then
// serves all but the first.
__device__ __forceinline__ const FewBlock *my_block(const int *plan, int &group)
{
    const FewBlock *list = (const FewBlock *)(plan + 4), *b = list + blockIdx.y;
    const int groups = (int)gridDim.x, of = b->of, first = b->first;
    group = (int)blockIdx.x;
    if ((int)blockIdx.y >= plan[0]) return nullptr;
    if (of > 1) {
        const int at = ((int)blockIdx.y - first) * groups + group, eight = at / (8 * of) * 8;
        const int n = min(8, groups - eight), i = at - eight * of;
        b = list + first + i / n;
        group = eight + i % n;
    }
    return b;
}

// silu_mul, but for NaNs: minima and maxima would make the clamp's limit of them.
__device__ __forceinline__ float gated(float gate, float up, float lim)
{
    const float v = silu_mul(gate, up, lim);
    return __builtin_isunordered(gate, up) ? __builtin_nanf("") : v;
}

template <int WT, int PATH, int WAVES>
__global__ __launch_bounds__(64 * WAVES, waves_per_simd(WT, WAVES)) void few_fc1_kernel(FewParams p, Layout l)
{
    extern __shared__ __align__(16) uint8_t lds[];
    int group;
    const FewBlock *blk = my_block(p.plan, group);
    if (!blk) return;
    const int e = blk->expert, row0 = blk->row0, m = blk->rows;
    const uintx4 tokens = *(const uintx4 *)blk->token;
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    block_product<WT, 1, PATH, WAVES>(
        lds, p.w1 + (int64_t)e * 2 * p.I * row_bytes(p.H, WT), p.w1s + (int64_t)e * 2 * p.I * (p.H / 32),
        Rows<1>{2 * p.I, p.I}, l, m, p.H, group,
        [&](int i) { return p.x + (int64_t)((tokens[i >> 2] >> (8 * (i & 3))) & 0xFFu) * p.H; },
        [&](int tile, floatx4 c) {
            *(bf16x2_t *)(p.h + (int64_t)(row0 + r) * p.I + tile * 8 + 2 * g) =
                bf16x2_t{(__bf16)gated(c[0], c[2], p.swiglu_limit), (__bf16)gated(c[1], c[3], p.swiglu_limit)};
        });
}

template <int WT, int PATH, int WAVES>
__global__ __launch_bounds__(64 * WAVES, waves_per_simd(WT, WAVES)) void few_fc2_kernel(FewParams p, Layout l)
{
    extern __shared__ __align__(16) uint8_t lds[];
    int group;
    const FewBlock *blk = my_block(p.plan, group);
    if (!blk) return;
    const int e = blk->expert, row0 = blk->row0, m = blk->rows;
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    block_product<WT, 2, PATH, WAVES>(
        lds, p.w2 + (int64_t)e * p.H * row_bytes(p.I, WT), p.w2s + (int64_t)e * p.H * (p.I / 32), Rows<2>{p.H, 0}, l, m,
        p.I, group, [&](int i) { return p.h + (int64_t)(row0 + i) * p.I; },
        [&](int tile, floatx4 c) {
            const int n0 = tile * kRows + 4 * g;
            if (n0 < p.H) *(floatx4 *)(p.y + (int64_t)(row0 + r) * p.H + n0) = c;
        });
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

int path_of(const void *w, int rb)
{
    if (((uintptr_t)w | (uintptr_t)rb) % 128) return kShared;
    return rb % 4096 ? kLines : kTurned;
}

template <int WT, int WAVES>
hipError_t launch_products(const FewParams &p, const Layout &l1, const Layout &l2, int cap, hipStream_t s)
{
    // the grid covers the most blocks the routing can give; the rest leave at once
    const int pairs = p.T * p.k, most = (p.E < pairs ? p.E : pairs) + pairs / cap;
    const unsigned blocks = (unsigned)(most < pairs ? most : pairs);
    const dim3 g1((unsigned)l1.groups, blocks), g2((unsigned)l2.groups, blocks), b(64 * WAVES);
    const int lds1 = l1.lds_fixed + cap * x_pitch(p.H, WT), lds2 = l2.lds_fixed + cap * x_pitch(p.I, WT);
    switch (path_of(p.w1, row_bytes(p.H, WT))) {
    case kTurned: hipLaunchKernelGGL((few_fc1_kernel<WT, kTurned, WAVES>), g1, b, lds1, s, p, l1); break;
    case kLines: hipLaunchKernelGGL((few_fc1_kernel<WT, kLines, WAVES>), g1, b, lds1, s, p, l1); break;
    default: hipLaunchKernelGGL((few_fc1_kernel<WT, kShared, WAVES>), g1, b, lds1, s, p, l1);
    }
    switch (path_of(p.w2, row_bytes(p.I, WT))) {
    case kTurned: hipLaunchKernelGGL((few_fc2_kernel<WT, kTurned, WAVES>), g2, b, lds2, s, p, l2); break;
    case kLines: hipLaunchKernelGGL((few_fc2_kernel<WT, kLines, WAVES>), g2, b, lds2, s, p, l2); break;
    default: hipLaunchKernelGGL((few_fc2_kernel<WT, kShared, WAVES>), g2, b, lds2, s, p, l2);
    }
    hipLaunchKernelGGL(few_sum_kernel, dim3((unsigned)((p.H / 4 + kThreads - 1) / kThreads), (unsigned)p.T),
                       dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_tokens(const FewParams &p, hipStream_t s)
{
    // The waves of a workgroup share its tokens' rows and its LDS.  Small workgroups hide each other's starts and end
    // evenly, which counts where little is read; large ones copy the tokens less often and hold more of them, and an
    // expert of more rows than they hold is read once for every block of them.  In us with 4, 8 and 16 waves: 1 token, 4
    // of 32 experts, 2880 x 2880 bf16: 45.4, 47.9, 54.6; 64 tokens, 6 of 256, 1056 x 544 4 bits: 62.7, 67.9, -; 40, 6 of
    // 256, 2016 x 992 4 bits: 93.7, 96.9, -; 24, 6 of 256, 4032 x 1984 4 bits: 224, 217, -; 5, 3 of 8, 4000 x 1952 bf16:
    // 62.7, 58.6, -; 33, 4 of 32, 2880 x 2880 8 bits: 155, 133, 145; 64, 6 of 8, 4032 x 1984 bf16 (8 waves: one workgroup
    // a CU): -, 236, 194.  The sums are the same.
    Layout l1, l2;
    const int pairs = p.T * p.k;
    const int64_t expert = 2 * (int64_t)p.I * row_bytes(p.H, p.weights) + (int64_t)p.H * row_bytes(p.I, p.weights);
    int cap = 0, waves = pairs <= 2 * p.E && pairs * expert <= (int64_t)1 << 30 ? 4 : 8;
    for (;; waves *= 2) {
        l1 = layout_of(p.I / 8, p.k, p.H, p.weights, waves);
        l2 = layout_of((p.H + kRows - 1) / kRows, p.k, p.I, p.weights, waves);
        const int per_cu = kCuWaves / waves;
        const int c1 = row_cap(l1, p.H, p.weights, p.T, per_cu), c2 = row_cap(l2, p.I, p.weights, p.T, per_cu);
        cap = c1 < c2 ? c1 : c2;
        // rows an expert may have on average; of 4 waves' LDS a third, since few tokens spread unevenly
        const int room = waves == 4 && cap < p.T ? p.E * cap / 3 : p.E * cap;
        if (waves == kCuWaves || (cap >= 1 && pairs <= room && l1.splits <= waves && l2.splits <= waves)) break;
    }
    hipError_t e = launch_moe_route_plan(p.route, RoutePlan{p.plan, cap}, s);
    if (e != hipSuccess) return e;
    const auto run = [&](auto wt) {
        constexpr int WT = decltype(wt)::value;
        switch (waves) {
        case 4: return launch_products<WT, 4>(p, l1, l2, cap, s);
        case 8: return launch_products<WT, 8>(p, l1, l2, cap, s);
        default: return launch_products<WT, kCuWaves>(p, l1, l2, cap, s);
        }
    };
    switch (p.weights) {
    case kFewMxfp8: return run(std::integral_constant<int, kFewMxfp8>{});
    case kFewMxfp4: return run(std::integral_constant<int, kFewMxfp4>{});
    default: return run(std::integral_constant<int, kFewBf16>{});
    }
}

}  // namespace ptgg
