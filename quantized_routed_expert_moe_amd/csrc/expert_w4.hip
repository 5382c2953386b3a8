// Expert products with 4-bit group-scaled weights: the streaming kernels of
// expert_stream.h at every row count (16, 32 or 64 rows a slot share one pass
// over the weights).
#include "expert_stream.h"

namespace qmoe {

hipError_t launch_expert_w4(const ExpertW4Args& a, hipStream_t s) {
    int shift = 5;
    while ((1 << shift) < a.group) ++shift;
    const StreamArgs t{a.x,   a.q, (size_t)a.N * (a.K / 2), a.scales, a.zeros, a.scale_dtype == MOE_F32, shift, a.N,
                       a.K,   a.rows, a.x_rows, a.y_rows, a.y, a.y_dtype == MOE_F32};
    return a.dtype == MOE_BF16 ? launch_stream_bf16(t, 1, a.act, s) : launch_stream_f16(t, 1, a.act, s);
}

}  // namespace qmoe
