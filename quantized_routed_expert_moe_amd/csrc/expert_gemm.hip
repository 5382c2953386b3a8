// Matrix products grouped by expert over ragged batches, and the weight
// gradient: the simple form, one output element per thread.
#include "expert_stream.h"

namespace qmoe {

// Slot that owns position q, or -1.
__device__ __forceinline__ int slot_of_position(const RowMap& m, int q) {
    if (!m.offsets) return 0;
    int lo = 0, hi = m.S;  // the last slot with offsets[slot] <= q
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (m.offsets[mid] <= q) lo = mid;
        else hi = mid;
    }
    const int2 r = slot_range(m, lo);
    return q >= r.x && q < r.x + r.y ? lo : -1;
}

template <int DT, int YT>
__global__ __launch_bounds__(256) void expert_gemm_simple(const ExpertGemmArgs a) {
    typedef typename DType<DT>::type E;
    const int q = blockIdx.y + gridDim.y * blockIdx.z;
    if (q >= a.rows.R) return;
    const int s = slot_of_position(a.rows, q);
    if (s < 0) return;
    const int in = a.transpose ? a.N : a.K;
    const int out = a.transpose ? a.K : a.act ? a.N / 2 : a.N;
    const E* x = static_cast<const E*>(a.x) + (size_t)row_of(a.rows, a.x_rows, q) * in;
    const E* w = reinterpret_cast<const E*>(static_cast<const uint8_t*>(a.w) + (size_t)s * a.w_stride);
    typename DType<YT>::type* y =
        static_cast<typename DType<YT>::type*>(a.y) + (size_t)row_of(a.rows, a.y_rows, q) * out;
    for (int c = blockIdx.x * 256 + threadIdx.x; c < out; c += gridDim.x * 256) {
        float v = 0.f, u = 0.f;
        if (a.transpose) {
            for (int n = 0; n < a.N; ++n) v = fmaf((float)x[n], (float)w[(size_t)n * a.K + c], v);
        } else {
            for (int j = 0; j < a.K; ++j) {
                v = fmaf((float)x[j], (float)w[(size_t)c * a.K + j], v);
                if (a.act) u = fmaf((float)x[j], (float)w[(size_t)(c + out) * a.K + j], u);
            }
            if (a.act) v = v * sigmoid_f32(v) * u;
        }
        y[c] = (typename DType<YT>::type)v;
    }
}

template <int DT, int YT>
__global__ __launch_bounds__(256) void expert_wgrad_simple(const ExpertWgradArgs a) {
    typedef typename DType<DT>::type E;
    const int s = blockIdx.z;
    const int2 r = slot_range(a.rows, s);
    const int j = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y;
    if (j >= a.K) return;
    float v = 0.f;
    for (int q = r.x; q < r.x + r.y; ++q)
        v = fmaf((float)static_cast<const E*>(a.dy)[(size_t)row_of(a.rows, a.dy_rows, q) * a.N + n],
                 (float)static_cast<const E*>(a.x)[(size_t)row_of(a.rows, a.x_rows, q) * a.K + j], v);
    static_cast<typename DType<YT>::type*>(a.dw)[((size_t)s * a.N + n) * a.K + j] = (typename DType<YT>::type)v;
}

hipError_t launch_expert_gemm(const ExpertGemmArgs& a, hipStream_t s) {
    if (a.rows.R == 0) return hipSuccess;
    const int slots = a.rows.offsets && a.rows.S < a.rows.R ? a.rows.S : a.rows.offsets ? a.rows.R : 1;
    if (!a.transpose && a.rows.R <= 32 * slots) {
        const StreamArgs t{a.x, a.w, a.w_stride, nullptr, nullptr, 0, 0, a.N, a.K, a.rows, a.x_rows, a.y_rows, a.y,
                           a.y_dtype == MOE_F32};
        return a.dtype == MOE_BF16 ? launch_stream_bf16(t, 0, a.act, s) : launch_stream_f16(t, 0, a.act, s);
    }
    const int out = a.transpose ? a.K : a.act ? a.N / 2 : a.N;
    const int gy = a.rows.R < 32768 ? a.rows.R : 32768;
    const dim3 grid((out + 255) / 256, gy, (a.rows.R + gy - 1) / gy);
    if (a.dtype == MOE_BF16) {
        if (a.y_dtype == MOE_F32) expert_gemm_simple<MOE_BF16, MOE_F32><<<grid, 256, 0, s>>>(a);
        else expert_gemm_simple<MOE_BF16, MOE_BF16><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.y_dtype == MOE_F32) expert_gemm_simple<MOE_F16, MOE_F32><<<grid, 256, 0, s>>>(a);
        else expert_gemm_simple<MOE_F16, MOE_F16><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

size_t expert_wgrad_workspace_bytes(int, int, int, int) { return 0; }

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t s) {
    const dim3 grid((a.K + 255) / 256, a.N, a.rows.S);
    if (a.dtype == MOE_BF16) {
        if (a.dw_dtype == MOE_F32) expert_wgrad_simple<MOE_BF16, MOE_F32><<<grid, 256, 0, s>>>(a);
        else expert_wgrad_simple<MOE_BF16, MOE_BF16><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.dw_dtype == MOE_F32) expert_wgrad_simple<MOE_F16, MOE_F32><<<grid, 256, 0, s>>>(a);
        else expert_wgrad_simple<MOE_F16, MOE_F16><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace qmoe
