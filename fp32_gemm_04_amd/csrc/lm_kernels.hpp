// The tile kernels that are built, by type, form and tile; shared by the
// host code (lm.hip) and the translation units that instantiate them.
#pragma once

#include "lm_rule.hpp"
#include "lm_tile.hpp"

namespace sgemm {
namespace lm {

struct TileKernel {
    TileFn fn;
    int bm, bn, threads;
};

// null fn: that tile is not built for the form and type (48 rows: fp32 only, and not
// where A's rows are contiguous in memory, since they make no whole 128-byte LDS rows).
TileKernel bf16_kernel(int form, int tile, bool fast);
TileKernel f32_kernel(int form, int tile, bool fast);

template <typename T, int BM, int BN, int WM, int WN, int NBUF, int BL, int WPE, bool FAST>
TileKernel tile_entry(int form)
{
    TileFn fn = nullptr;
    switch (form) {
    case F_ROWS_T: fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, KC, KC, ROWS, STORE, FAST>; break;
    case F_ROWS_N: fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, KC, MC, ROWS, STORE, FAST>; break;
    case F_SUM:
        if constexpr (BM != 48) fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, MC, MC, SUM, STORE, FAST>;
        break;
    case F_STATS: fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, KC, KC, PLAIN, STATS, FAST>; break;
    case F_GRAD: fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, KC, KC, PLAIN, GRAD, FAST>; break;
    case F_PART: fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, KC, MC, PLAIN, PART, FAST>; break;
    case F_DX: fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, KC, MC, PLAIN, STORE, FAST>; break;
    case F_DW:
        if constexpr (BM != 48) fn = tile_kernel<T, BM, BN, WM, WN, NBUF, BL, WPE, MC, MC, PLAIN, STORE, FAST>;
        break;
    default: break;
    }
    return TileKernel{fn, BM, BN, WM * WN * 64};
}

}  // namespace lm
}  // namespace sgemm
