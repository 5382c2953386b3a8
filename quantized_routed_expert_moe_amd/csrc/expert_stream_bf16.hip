// The streaming expert products of bf16 rows (expert_stream.h).
#include "expert_stream.h"

namespace qmoe {
hipError_t launch_stream_bf16(const StreamArgs& a, int w4, int act, hipStream_t s) {
    return stream_launch_type<MOE_BF16>(a, w4, act, s);
}
}  // namespace qmoe
