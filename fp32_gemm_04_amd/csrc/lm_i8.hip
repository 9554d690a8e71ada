// 8-bit integer tile kernels of the language-model products.
#include "lm_kernels.hpp"

namespace sgemm {
namespace lm {

namespace {

template <typename TC, int BM, int BN, int WM, int WN, int NBUF, int BL, int WPE, bool FAST>
TileKernel entry(bool grouped)
{
    return TileKernel{
        grouped
            ? (TileFn)tile_kernel<int8_t, BM, BN, WM, WN, NBUF, BL, WPE, KC, KC, ROWS, SCALE, FAST, TC>
            : (TileFn)tile_kernel<int8_t, BM, BN, WM, WN, NBUF, BL, WPE, KC, KC, PLAIN, SCALE, FAST, TC>,
        BM, BN, WM * WN * 64};
}

template <typename TC>
TileKernel of_type(bool grouped, int tile, bool fast)
{
    if (!fast) {
        if (tile == M32) return entry<TC, 32, 128, 1, 4, 2, 16, 2, false>(grouped);
        if (tile == M64) return entry<TC, 64, 128, 2, 2, 2, 16, 2, false>(grouped);
        return entry<TC, 128, 128, 2, 2, 2, 16, 2, false>(grouped);
    }
    switch (tile) {
    case M64: return entry<TC, 64, 128, 2, 2, 3, 16, 2, true>(grouped);
    case T128: return entry<TC, 128, 128, 2, 2, 2, 16, 2, true>(grouped);
    case T192: return entry<TC, 128, 192, 2, 2, 2, 16, 2, true>(grouped);
    default: return entry<TC, 256, 256, 2, 2, 2, 32, 1, true>(grouped);
    }
}

}  // namespace

TileKernel i8_kernel(bool bf16_out, bool grouped, int tile, bool fast)
{
    return bf16_out ? of_type<bf16>(grouped, tile, fast) : of_type<float>(grouped, tile, fast);
}

}  // namespace lm
}  // namespace sgemm
