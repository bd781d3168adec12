// The tiles of linear_tile.h for FP16 operands.
#include <type_traits>

#include "linear_tile.h"

int misgemm_linear::launch_tiles_f16(bool gated, bool ta, bool tb, int shape, LinArgs &g, hipStream_t stream) {
    return launch_tiles<f16>(gated, ta, tb, shape, g, stream);
}
