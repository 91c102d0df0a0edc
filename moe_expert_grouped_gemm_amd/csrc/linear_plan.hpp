// linear_plan.hpp -- how a dense product runs: which tile, and in how many parts.
// Host code, from sizes alone; a host build of it checks that the parts cover a
// product.
#pragma once
#include "dense.hpp"

namespace ptgg {
namespace {

constexpr int kWide = 256;                    // rows and columns of the widest tile
constexpr int kStage = 64;                    // reduction values of a stage

// The tiles, with what a call of theirs costs in us: `fixed` (launch, first loads,
// epilogue) and a stage of 64 reduction values while a CU holds one workgroup and,
// where two fit, while it holds two.  Fitted to forward products of 1021 x 2880 x
// 2880, 45 to 4096 x 4096 x 4096 and slices of their reduction; the other layouts
// take up to a fifth longer, alike for all tiles.  The deep ones keep a CU's LDS for
// one workgroup's ring, which pays where there are too few tiles for two.
// Costs of whole calls, to rank tiles by: of large products they are near what is
// measured (8192^3 727 us for 705, 4096^3 100 for 95), of smaller ones above it (4096
// x 2880 x 2880 73 for 59, 2048 53 for 38, 1021 32 for 23, 512 25 for 17; 45 x 4096 x
// 4096 16.5 for 13.2), and where memory is the bound, which they do not know, below
// (65536 x 64 x 2880 53 for 80).  So near a border between two tiles the choice may
// not be the faster one.
enum Tile {
    kTileFew = 0, kTile256 = 1, kTile128 = 2, kTile64 = 3, kTileNarrow = 4, kTile128Deep = 5, kTile64Deep = 6, kTile32Deep = 7
};
struct TileShape {
    int tm, tn, per_cu;
    float fixed, stage1, stage2;
};
// from kTile256 on
constexpr TileShape kTiles[] = {{256, 256, 1, 10.0f, 1.40f, 1.40f},
                                {128, 128, 2, 8.0f, 0.78f, 1.00f},
                                {64, 128, 2, 6.5f, 0.41f, 0.70f},
                                {64, 32, 2, 7.0f, 0.25f, 0.35f},
                                {128, 128, 1, 8.0f, 0.54f, 0.54f},
                                {64, 128, 1, 6.8f, 0.40f, 0.40f},
                                {32, 128, 1, 6.5f, 0.36f, 0.36f}};
constexpr int kCus = 256;
constexpr float kJoin = 3.2f, kPartialRate = 5e6f;      // us of the join's launch; bytes a us of partial sums

// Tiles of the widest kind over the CUs, one to a CU at a time.  Whole tiles fill all
// CUs some times over; the r that are left would keep r of them busy as long again.
// So their reduction is cut: p = G / r parts a tile, and the e CUs that this leaves
// take the tiles' tails, f of them one after another, and then what is left of the
// tails in pieces: a tail is as long as lets both kinds of CUs end together.  Pieces
// of a kind start at the same places of the reduction, so that an XCD's L2 serves
// its tiles' common rows once.  Parts and pieces are at least about as long as their
// start and end (16384 x 2880 x 2880 wgrad: 260 us, three equal parts 286; 8192 x
// 2880 x 11520: 401, whole tiles 445).
inline WideCut wide_cut(int tiles, int stages)
{
    constexpr float kPiece = 8.0f;                       // a piece's start and end, in stages (23000 cycles)
    WideCut cut = {tiles, 0, 0, 0, 0, 0, 0};
    const int r = tiles % kCus;
    if (r == 0) return cut;
    const int fit = kCus / r, p = min(fit, max(stages / 8, 1)), e = p < fit ? 0 : kCus - p * r;
    int tail = 0, f = 0, c = 1;
    if (e > 0) {
        f = r / e;
        const int left = r - f * e;
        c = left ? max(e / left, 1) : 1;
        // main = slope tail + extra, stages = p main + tail
        const float slope = (float)f + (left ? 1.0f / (float)c : 0.0f), extra = (float)(f + (left ? 1 : 0) - 1) * kPiece;
        const float x = ((float)stages - (float)p * extra) / (1.0f + (float)p * slope);
        tail = x >= 4.0f ? (int)x : 0;
    }
    const int main = (stages - tail + p - 1) / p;
    tail = stages - p * main;
    if (tail <= 0 && p == 1) return cut;
    cut.whole = tiles - r;
    cut.rest = r;
    cut.main = (int64_t)main * kStage;
    if (tail <= 0) {
        cut.parts = (stages + main - 1) / main;
        return cut;
    }
    cut.parts = p;
    cut.tails = f * e;
    c = min(c, max(tail / 8, 1));
    const int piece = (tail + c - 1) / c;
    cut.cuts = (tail + piece - 1) / piece;
    cut.cut = (int64_t)piece * kStage;
    return cut;
}

// Up to 16 rows w streams through the few-row kernel (1 x 4096 x 4096: 10.5 us, 12.7
// by tiles; 16: 13.3 and 13.3; since then 9.7 and 12.3, 17 by tiles 12.4).  Else the
// tile and the parts of the reduction whose cost by the table above is least, of the
// narrow tile up to the 32 columns that one of them holds (16384 x 32 x 2880: 21.4 us,
// 24.3 by the others).  Beyond, two of them lose or win: 16384 x 64 x 2880 28.4 us,
// 25.3 by the tile chosen, 40 columns 25.9 and 23.6; 8192 x 64 x 4096 18.4 and 20.7,
// 2000 x 64 x 2880 9.7 and 10.9.
inline LinearPlan plan_linear(int op, int64_t M, int64_t N, int64_t K)
{
    LinearPlan best = {kTileFew, 1, (K + kStage - 1) / kStage * kStage, {}, 0};
    if (op == kLinFwd && M <= 16) return best;
    const int stages = (int)((K + kStage - 1) / kStage);                  // at most 2^17
    float cost = 0;
    for (int t = kTile256; t <= kTile32Deep; ++t) {
        const TileShape &sh = kTiles[t - kTile256];
        if (t == kTileNarrow ? op != kLinFwd || N > 32 : t == kTile32Deep && op == kLinWgrad) continue;
        const int64_t all = ((M + sh.tm - 1) / sh.tm) * ((N + sh.tn - 1) / sh.tn);
        if (t != kTile256 && all > (1 << 22)) continue;                  // a launch holds 2^32 threads
        const int tiles = (int)all, full = kCus * sh.per_cu;
        if (t == kTile256) {
            const WideCut whole = {tiles, 0, 0, 0, 0, 0, 0}, cut = wide_cut(tiles, stages);
            cost = (float)((tiles + kCus - 1) / kCus) * (float)stages * sh.stage1 + sh.fixed;
            best = {t, 1, 0, whole, 0};
            if (cut.rest) {
                const float c = ((float)(tiles / kCus) * (float)stages + (float)(cut.main / kStage)) * sh.stage1 + sh.fixed + kJoin +
                                (float)cut.pieces() * (kWide * kWide * 8.0f / kPartialRate);
                if (c < cost) cost = c, best = {t, 1, 0, cut, (int64_t)cut.pieces() * kWide * kWide * 4};
            }
            continue;
        }
        for (const int want : {1, 2, 3, 4, 5, 6, 8, 12, 16, 24, 32, 64}) {
            if (want > 1 && (tiles > 4 * kCus / want || stages < 2 * want)) break;
            const int per = stages > 0 ? (stages + want - 1) / want : 1, splits = stages > 0 ? (stages + per - 1) / per : 1;
            const int wgs = tiles * splits, rounds = wgs / full, rest = wgs - rounds * full;
            float c = (float)rounds * sh.stage2;
            if (rest) c += rest <= kCus ? sh.stage1 : sh.stage2;
            c = c * (float)per + sh.fixed;
            if (splits > 1) c += kJoin + (float)splits * ((float)(M * N) * (8.0f / kPartialRate) + 0.15f);
            if (c < cost) {
                cost = c;
                best = {t, splits, (int64_t)per * kStage, {}, splits > 1 ? splits * M * N * 4 : 0};
            }
        }
    }
    return best;
}

}  // namespace
}  // namespace ptgg
