// The tiled expert products of fp16 rows (expert_tile.h).
#include "expert_tile.h"

namespace qmoe {
hipError_t launch_tile_f16(const TileArgs& a, int mode, int act, int big, hipStream_t s) {
    return tile_launch_type<MOE_F16>(a, mode, act, big, s);
}
}  // namespace qmoe
