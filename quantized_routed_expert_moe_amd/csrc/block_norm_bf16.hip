// The block norms of bf16 rows (block_norm.h).
#include "block_norm.h"

namespace qmoe {
void norm_launch_bf16(const BlockNormArgs& a, int backward, dim3 grid, hipStream_t s) {
    norm_launch_type<MOE_BF16>(a, backward, grid, s);
}
}  // namespace qmoe
