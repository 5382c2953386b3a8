// Expert products with 4-bit group-scaled weights: the simple form, one
// output element per thread.
#include "expert_ops.h"

namespace qmoe {

template <int DT, int YT>
__global__ __launch_bounds__(256) void expert_w4_simple(const ExpertW4Args a) {
    typedef typename DType<DT>::type E;
    const int s = blockIdx.z;
    const int2 r = slot_range(a.rows, s);
    const int out = a.act ? a.N / 2 : a.N, G = a.K / a.group;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= out) return;
    for (int q = r.x + blockIdx.y; q < r.x + r.y; q += gridDim.y) {
        const E* x = static_cast<const E*>(a.x) + (size_t)row_of(a.rows, a.x_rows, q) * a.K;
        float v[2] = {0.f, 0.f};
        for (int m = 0; m < (a.act ? 2 : 1); ++m) {
            const size_t row = (size_t)s * a.N + c + m * out;
            for (int g = 0; g < G; ++g) {
                const float sc = a.scale_dtype == MOE_F32 ? static_cast<const float*>(a.scales)[row * G + g]
                                                          : (float)static_cast<const E*>(a.scales)[row * G + g];
                const float z = a.zeros ? (float)a.zeros[row * G + g] : 8.f;
                float t = 0.f;
                for (int j = g * a.group; j < (g + 1) * a.group; ++j) {
                    const int b = a.q[row * (a.K / 2) + j / 2];
                    t = fmaf((float)(j & 1 ? b >> 4 : b & 15) - z, (float)x[j], t);
                }
                v[m] = fmaf(sc, t, v[m]);
            }
        }
        const float o = a.act ? v[0] * sigmoid_f32(v[0]) * v[1] : v[0];
        static_cast<typename DType<YT>::type*>(a.y)[(size_t)row_of(a.rows, a.y_rows, q) * out + c] =
            (typename DType<YT>::type)o;
    }
}

hipError_t launch_expert_w4(const ExpertW4Args& a, hipStream_t s) {
    if (a.rows.R == 0) return hipSuccess;
    const int out = a.act ? a.N / 2 : a.N;
    const dim3 grid((out + 255) / 256, a.rows.R < 64 ? a.rows.R : 64, a.rows.S);
    if (a.dtype == MOE_BF16) {
        if (a.y_dtype == MOE_F32) expert_w4_simple<MOE_BF16, MOE_F32><<<grid, 256, 0, s>>>(a);
        else expert_w4_simple<MOE_BF16, MOE_BF16><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.y_dtype == MOE_F32) expert_w4_simple<MOE_F16, MOE_F32><<<grid, 256, 0, s>>>(a);
        else expert_w4_simple<MOE_F16, MOE_F16><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace qmoe
