// fp32 tile kernels of the language-model products.
#include "lm_kernels.hpp"

namespace sgemm {
namespace lm {

TileKernel f32_kernel(int form, int tile, bool fast)
{
    if (!fast) {
        if (tile == S16) return tile_entry<float, 16, 64, 1, 4, 2, 16, 2, false>(form);
        if (tile == M32) return tile_entry<float, 32, 64, 1, 4, 2, 16, 2, false>(form);
        if (tile == M64) return tile_entry<float, 64, 64, 2, 2, 2, 16, 2, false>(form);
        return tile_entry<float, 128, 128, 2, 2, 2, 16, 2, false>(form);
    }
    switch (tile) {
    case S16: return tile_entry<float, 16, 64, 1, 4, 4, 16, 4, true>(form);
    case M32: return tile_entry<float, 32, 64, 1, 4, 4, 16, 3, true>(form);
    case M64: return tile_entry<float, 64, 64, 2, 2, 3, 16, 2, true>(form);
    default: return tile_entry<float, 128, 128, 2, 2, 2, 16, 2, true>(form);
    }
}

}  // namespace lm
}  // namespace sgemm
