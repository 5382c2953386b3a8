// The streamed biased products of bf16 rows (expert_stream.h).
#include "expert_stream.h"

namespace qmoe {
hipError_t launch_stream_bias_bf16(const StreamArgs& a, int act, hipStream_t s) {
    return stream_launch<0, MOE_BF16, 4, true>(a, act, s);
}
}  // namespace qmoe
