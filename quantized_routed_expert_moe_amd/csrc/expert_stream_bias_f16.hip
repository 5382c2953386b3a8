// The streamed biased products of fp16 rows (expert_stream.h).
#include "expert_stream.h"

namespace qmoe {
hipError_t launch_stream_bias_f16(const StreamArgs& a, int act, hipStream_t s) {
    return stream_launch<0, MOE_F16, 4, true>(a, act, s);
}
}  // namespace qmoe
