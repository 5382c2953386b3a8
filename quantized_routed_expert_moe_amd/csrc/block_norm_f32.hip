// The block norms of fp32 rows (block_norm.h).
#include "block_norm.h"

namespace qmoe {
void norm_launch_f32(const BlockNormArgs& a, int backward, dim3 grid, hipStream_t s) {
    norm_launch_type<MOE_F32>(a, backward, grid, s);
}
}  // namespace qmoe
