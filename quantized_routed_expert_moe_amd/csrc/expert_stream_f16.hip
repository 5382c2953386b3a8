// The streaming expert products of fp16 rows (expert_stream.h).
#include "expert_stream.h"

namespace qmoe {
hipError_t launch_stream_f16(const StreamArgs& a, int w4, int act, hipStream_t s) {
    return stream_launch_type<MOE_F16>(a, w4, act, s);
}
}  // namespace qmoe
