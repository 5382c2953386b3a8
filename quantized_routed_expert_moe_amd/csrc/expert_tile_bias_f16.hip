// The tiled biased products of fp16 rows (expert_tile.h).
#include "expert_tile.h"

namespace qmoe {
hipError_t launch_tile_bias_f16(const TileArgs& a, int act, int big, hipStream_t s) {
    return tile_launch_bias<MOE_F16>(a, act, big, s);
}
}  // namespace qmoe
