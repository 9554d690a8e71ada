// fp32 tile kernels of the language-model products.
#include "lm_kernels.hpp"

namespace sgemm {
namespace lm {

TileKernel f32_kernel(int form, int tile, bool fast)
{
    if (!fast) {
        if (tile == S16) return tile_entry<float, 16, 64, 1, 4, 2, 16, 2, false>(form);
        if (tile == M32) return tile_entry<float, 32, 64, 1, 4, 2, 16, 2, false>(form);
        if (tile == M48) return tile_entry<float, 48, 128, 1, 4, 2, 16, 2, false>(form);
        if (tile == M64) return tile_entry<float, 64, 64, 2, 2, 2, 16, 2, false>(form);
        return tile_entry<float, 128, 128, 2, 2, 2, 16, 2, false>(form);
    }
    // Buffers and workgroups on a unit: where a unit has one tile, a deeper ring hides the
    // latency of memory; where it has many, more workgroups do.  48 x 128, H 1024, V 32000:
    // T 37 (250 tiles) 46.5 us with two buffers and three workgroups, 39.6 with three and
    // two, 40.4 with four and one; T 140 83.9, 90.1 and 105.  64 x 64: the backward pass of
    // 24 experts' 1500 rows 45.7 us with two and four, 48 with three and two.
    switch (tile) {
    case S16: return tile_entry<float, 16, 64, 1, 4, 4, 16, 4, true>(form);
    case M32: return tile_entry<float, 32, 64, 1, 4, 4, 16, 3, true>(form);
    case M48: return tile_entry<float, 48, 128, 1, 4, 3, 16, 2, true>(form);
    case M64: return tile_entry<float, 64, 64, 2, 2, 2, 16, 4, true>(form);
    default: return tile_entry<float, 128, 128, 2, 2, 2, 16, 2, true>(form);
    }
}

}  // namespace lm
}  // namespace sgemm
