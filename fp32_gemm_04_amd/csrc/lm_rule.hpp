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
