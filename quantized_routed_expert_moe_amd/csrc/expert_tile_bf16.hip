// The tiled expert products of bf16 rows (expert_tile.h).
#include "expert_tile.h"

namespace qmoe {
hipError_t launch_tile_bf16(const TileArgs& a, int mode, int act, int big, hipStream_t s) {
    return tile_launch_type<MOE_BF16>(a, mode, act, big, s);
}
}  // namespace qmoe
