// Which tile a language-model product runs with, and how the cross entropy's backward pass
// is cut: rules on sizes alone, in plain C++.
#pragma once

#include <cstdint>

#include "lm_host.hpp"

namespace sgemm {
namespace lm {

enum Tile { S16, M32, M48, M64, T128, T192, T256, NUM_TILES };
// The operand layouts and epilogues of the products.
enum Form {
    F_ROWS_T,   // grouped rows, weights N x K
    F_ROWS_N,   // grouped rows, weights K x N
    F_SUM,      // grouped contraction
    F_STATS,    // logits to row statistics
    F_GRAD,     // logits to their derivatives
    F_PART,     // d W, fp32 sums
    F_DX,       // d W, rounded to the type
    F_DW,       // d^T X
    NUM_FORMS
};

// What a tile costs: outputs times contraction over `rate`, the rate its kernel reaches
// on a compute unit relative to the largest tile's, `lead` being the contraction's worth
// of time that filling the ring and writing the tile take when nothing else runs on the
// unit (the 256 tile leaves no room for a second workgroup).  Measured, bf16: T 8192, H 2048, V
// 131072 with gradients 15.9 ms with the 256 tile, 16.9 with 128 x 192; T 384, H 1024, V
// 50021 369 and 277 us; 16 experts' backward pass of 16384 rows 381 and 349 us (128 x
// 128: 403, 64 x 128: 477).  fp32: T 1023, H 1000, V 49999 3.22 ms with the 128 tile,
// 3.35 with 64 x 64; 24 experts' backward pass of 1500 rows 93 and 63 us; the loss of 37
// rows (H 1024, V 32000) 45.9 us with 64 x 64 and 39.6 with 48 x 128, of 140 rows 114 and 90.
struct TileCost {
    int bm, bn;
    double rate;
    int lead;
};
constexpr TileCost kBf16Tiles[NUM_TILES] = {
    {16, 64, 0.2, 64}, {32, 128, 0.45, 64}, {0, 0, 0, 0}, {64, 128, 0.65, 64}, {128, 128, 0.8, 64}, {128, 192, 0.88, 64},
    {256, 256, 1.0, 256}};
constexpr TileCost kF32Tiles[NUM_TILES] = {
    {16, 64, 0.5, 64}, {32, 64, 0.75, 64}, {48, 128, 0.9, 64}, {64, 64, 0.87, 64}, {128, 128, 1.0, 64}, {0, 0, 0, 0}, {0, 0, 0, 0}};

// By the size of an element.
inline const TileCost *tile_costs(int size) { return size == 2 ? kBf16Tiles : kF32Tiles; }

// The tile that finishes first when every compute unit takes the same number of tiles
// (a last one that has the unit to itself counts half where two fit beside each other):
// products of N columns and contraction K, whose rows split into row_tiles(bm) tiles in
// all.
template <typename RowTiles>
int choose_tile(int size, int form, bool fast, RowTiles row_tiles, int64_t N, int64_t K, int cus)
{
    const TileCost *t = tile_costs(size);
    int best = S16;
    double least = 0;
    for (int i = 0; i < (fast ? (int)NUM_TILES : T128 + 1); ++i) {
        if (t[i].bm == 0 || (i == M48 && (form == F_SUM || form == F_DW))) continue;
        const int64_t tiles = row_tiles(t[i].bm) * ceil_div(N, t[i].bn);
        const bool pairs = t[i].lead == 64 && tiles > cus;
        const double rounds = pairs ? 0.5 * ceil_div(2 * tiles, cus) : (double)ceil_div(tiles, cus);
        const double cost = rounds * t[i].bm * t[i].bn * (K + t[i].lead) / t[i].rate;
        if (i == 0 || cost < least) best = i, least = cost;
    }
    return best;
}

// For one product of M x N outputs.
inline int plain_tile(int size, int form, bool fast, int64_t M, int64_t N, int64_t K, int cus)
{
    return choose_tile(size, form, fast, [&](int bm) { return ceil_div(M, bm); }, N, K, cus);
}

// For rows that fall into groups, `used` of them not empty at most; a group's last tile is
// half full on average.
inline int rows_tile(int size, bool fast, int64_t used, int64_t rows, int64_t N, int64_t K, int cus)
{
    const auto row_tiles = [&](int bm) {
        const int64_t t = rows / bm + used / 2;
        return t > used ? t : used;
    };
    return choose_tile(size, F_ROWS_N, fast, row_tiles, N, K, cus);
}

// 8-bit products.  As above, with the contraction in pairs of bytes (a slab is 64); a unit takes two
// tiles at a time (of the 256 tile one), and where a last one has the unit to itself it costs
// `alone`, in tiles of a unit that is never idle.  Rates are those of 8192 x 4096 x 14336 (439 us
// with the 256 tile; 479, 557 and 657 us with the smaller ones).  Small tiles have the contraction split over
// waves: there time goes with the bytes of both operands.  alone and lead were fitted to the times of all on
// 86 sizes of 17 to 32768 rows, and the split ones' to 390 sizes of 1 to 8192: the rule's choice is 1.5%
// slower than the best of these on average, 1.8% on 130 sizes from 300 rows on.  Of 13 kernels the six
// tiles without the split ones are 20.6% slower, with one, two and three of them 3.6, 1.6 and 0.9%, each
// choice the best there is.  Operands without direct loads have costs of their own, fitted to 180 sizes (2.7%;
// 18.2% without the split ones, which take more registers from 32 x 64 on than there are).
struct ByteTileCost {
    int bm, bn;
    double rate, alone;
    int lead;
};
constexpr int kSplits = 4;
constexpr ByteTileCost kI8Tiles[2][NUM_TILES] = {
    {{}, {32, 128, 0.576, 1.18, 400}, {}, {64, 128, 0.667, 1.51, 150}, {128, 128, 0.829, 1.55, 207}, {}, {}},
    {{}, {}, {}, {64, 128, 0.67, 1.55, 128}, {128, 128, 0.79, 1.4, 96}, {128, 192, 0.92, 1.65, 64},
     {256, 256, 1.0, 0.9, 128}}};
constexpr ByteTileCost kI8Splits[2][kSplits] = {
    {{16, 32, 0.0429, 0.92, 700}, {32, 32, 0.0637, 1.41, 1340}, {}, {}},
    {{16, 32, 0.0321, 0.71, 1152}, {32, 32, 0.0295, 0.82, 1152}, {32, 64, 0.0264, 0.71, 832},
     {64, 64, 0.026, 0.71, 1408}}};

// Workgroups of a product with bm x bn tiles: of rows of one group (used 0), or of `used` groups, whose
// last tiles may be part full.
inline int64_t byte_blocks(int64_t used, int64_t rows, int64_t N, int bm, int bn)
{
    return (rows + (used ? used : 1) * (bm - 1)) / bm * ceil_div(N, bn);
}
// Sides of the largest tile.
constexpr int byte_side(bool fast) { return fast ? 256 : 128; }

// A tile, or NUM_TILES and which of the split ones, whose workgroups one launch takes (fits); -1: there is none.
template <typename RowTiles, typename Fits>
int byte_tile(bool fast, RowTiles row_tiles, Fits fits, int64_t N, int64_t K, int cus)
{
    int best = -1;
    double least = 0;
    const auto offer = [&](int i, const ByteTileCost &t, double cost) {
        if ((best < 0 || cost < least) && fits(t.bm, t.bn)) best = i, least = cost;
    };
    for (int i = 0; i < NUM_TILES; ++i) {
        const ByteTileCost &t = kI8Tiles[fast][i];
        if (t.bm == 0) continue;
        const int64_t tiles = row_tiles(t.bm) * ceil_div(N, t.bn);
        const int64_t left = tiles % (2 * cus);
        double rounds = (double)(tiles / (2 * cus)) * 2 + (left == 0 ? 0 : left <= cus ? t.alone : 2);
        if (i == T256) rounds = tiles <= cus ? t.alone : (double)ceil_div(tiles, cus);
        offer(i, t, rounds * t.bm * t.bn * (0.5 * K + t.lead) / t.rate);
    }
    for (int i = 0; i < kSplits; ++i) {
        const ByteTileCost &t = kI8Splits[fast][i];
        if (t.bm == 0) continue;
        const double share = (double)(row_tiles(t.bm) * ceil_div(N, t.bn)) / cus;
        offer(NUM_TILES + i, t, (share > t.alone ? share : t.alone) * (t.bm + t.bn) * (K + t.lead) / t.rate);
    }
    return best;
}

// For rows of one group (groups 0) or of `used` groups.
inline int byte_rows_tile(bool fast, int64_t used, int64_t rows, int64_t N, int64_t K, int cus)
{
    const auto row_tiles = [&](int bm) {
        if (used == 0) return ceil_div(rows, bm);
        const int64_t t = rows / bm + used / 2;
        return t > used ? t : used;
    };
    const auto fits = [&](int bm, int bn) { return byte_blocks(used, rows, N, bm, bn) <= kMostBlocks; };
    return byte_tile(fast, row_tiles, fits, N, K, cus);
}

// Whether rows of one group (groups 0), or of `used` of the groups, are few enough for a workgroup to hold
// them while it streams weights.  us, that and the best of the others: direct loads of one group, 1 row,
// 4096 x 4096 5.4 and 5.7, 16 rows 8.3 and 5.7, 12 rows, 8192 x 28001 48.4 and 42.1; by group, 16 rows, 4 groups
// of 2048 x 1536 5.8 and 5.3, 29 rows, 12 groups of 1136 x 1561 8.9 and 8.5, but 64 rows, 256 groups
// of 2048 x 1408, each tile of which is found by counting all of them, 29.2 and 33.8.
inline bool byte_few_rows(bool fast, int64_t groups, int64_t used, int64_t rows)
{
    if (fast && groups <= 64) return false;
    return groups <= 65535 && rows <= (groups ? 4 * used : 16);
}

// For M x N outputs of each group, the contraction over its rows.
inline int sum_tile(int size, bool fast, int groups, int rows, int64_t M, int64_t N, int cus)
{
    const auto row_tiles = [&](int bm) { return ceil_div(M, bm) * groups; };
    return choose_tile(size, F_SUM, fast, row_tiles, N, rows / groups, cus);
}

// How the backward pass is cut: `piece` columns of the vocabulary at a time, and
// the sum over a piece that gives dX in `slices` (few rows and hidden values
// leave compute units idle otherwise).
struct XentPlan {
    int64_t piece, pieces, ld;  // ld: leading dimension of the piece's derivatives
    int slices, dx_tile, dx_form;
    int low_rows, d_rows;       // rows to the rounding's remainders (0: not kept); rows in all
    bool sums;                  // dX goes through fp32 sums in the workspace
    int64_t d_bytes, bytes;
};

// Every extent at least 1.
inline XentPlan xent_plan(int size, bool fast, int rows, int vocab, int K, int cus)
{
    XentPlan p;
    // A piece's derivatives take up to 256 MiB (the last-level cache's size), but a
    // piece is never narrower than 2048 columns.
    int64_t most = ((int64_t)256 << 20) / ((int64_t)rows * size) / 256 * 256;
    if (most < 2048) most = 2048;
    if (most > (1 << 20) - 256) most = (1 << 20) - 256;  // fast_operand's limit for its rows
    p.pieces = ceil_div(vocab, most);
    p.piece = round_up(ceil_div(vocab, p.pieces), 256);
    p.pieces = ceil_div(vocab, p.piece);
    p.ld = p.piece + 64;
    // A row's gradient is mostly one derivative's (its target's), whose rounding to bf16
    // shifts the whole row by up to 2^-8 (one row: 0.0034 off, against 0.0017 of an fp32 sum
    // rounded once).  With few rows, where the time is that of reading W and writing dW, what
    // the rounding leaves over is kept as further rows.  With many it would double the
    // products' work, so each derivative is rounded, as a stored gradient of the type would
    // be (T 384: 0.0022 off), also where all round the same way, as with one dloss in all
    // rows.
    p.low_rows = size != 2 || rows > 128 ? 0
                 : rows <= 8             ? 8
                 : rows <= 16            ? 16
                 : rows <= 32            ? 32
                                         : (int)round_up(rows, 64);
    p.d_rows = p.low_rows ? 2 * p.low_rows : rows;
    p.d_bytes = round_up((int64_t)p.d_rows * p.ld * size, 256);
    // dX may have few tiles and a long sum: where its tiles would not fill the compute
    // units, the tile is chosen as if the sum were cut as finely as it may be (1024
    // columns a slice), and cut until each unit has two.
    const int64_t most_slices = p.piece / 1024 < 1 ? 1 : p.piece / 1024 > 64 ? 64 : p.piece / 1024;
    p.dx_tile = plain_tile(size, F_PART, fast, p.d_rows, K, p.piece, cus);
    p.slices = 1;
    if (ceil_div(p.d_rows, 128) * ceil_div(K, 128) < cus) {
        p.dx_tile = choose_tile(
            size, F_PART, fast, [&](int bm) { return ceil_div(p.d_rows, bm) * most_slices; }, K,
            p.piece / most_slices, cus);
        const TileCost &t = tile_costs(size)[p.dx_tile];
        const int64_t s = 2 * cus / (ceil_div(p.d_rows, t.bm) * ceil_div(K, t.bn));
        p.slices = (int)(s < 1 ? 1 : s > most_slices ? most_slices : s);
    }
    p.sums = p.low_rows > 0 || p.slices > 1 || (p.pieces > 1 && size != 4);
    p.dx_form = p.sums || p.pieces > 1 ? F_PART : F_DX;
    p.bytes = p.d_bytes + (p.sums ? (int64_t)p.slices * p.d_rows * K * 4 : 0);
    return p;
}

// For the derivatives of a piece of n columns.
inline int grad_tile(int size, bool fast, const XentPlan &p, int rows, int64_t n, int64_t K, int cus)
{
    const int tile = plain_tile(size, F_GRAD, fast, p.low_rows ? p.low_rows : rows, n, K, cus);
    return p.low_rows && tile == T256 ? (int)T192 : tile;  // the 256 tile keeps no remainders
}

// Each row's value at its target, and its statistics over the columns of each tile, of
// the narrower of the tiles that run with and without direct loads.
inline int64_t stats_bytes(int size, int rows, int vocab, int K, int cus)
{
    const TileCost *t = tile_costs(size);
    const int a = t[plain_tile(size, F_STATS, true, rows, vocab, K, cus)].bn;
    const int b = t[plain_tile(size, F_STATS, false, rows, vocab, K, cus)].bn;
    return round_up((int64_t)rows * 4, 256) + (int64_t)rows * ceil_div(vocab, a < b ? a : b) * 8;
}

}  // namespace lm
}  // namespace sgemm
