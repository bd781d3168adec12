// The tiles of linear_tile.h for BF16 operands.
#include <type_traits>

#include "linear_tile.h"

int misgemm_linear::launch_tiles_bf16(bool gated, bool ta, bool tb, int shape, LinArgs &g, hipStream_t stream) {
    return launch_tiles<bf16>(gated, ta, tb, shape, g, stream);
}
