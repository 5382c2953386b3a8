// The weighted combine's gradients: dy_pairs[p] = w_p dy[t] and dw[p] = <y_pairs[p], dy[t]>.
//
// Bound by HBM: each pair's row is read and one written, a token's row of dy read.
// A workgroup owns a token's pairs, eight at a time: a thread holds eight columns of
// dy and takes them through the eight pairs, whose loads are in flight together, and
// the eight sums are joined in wave order at the end.
#include "train_ops.h"

namespace qmoe {

constexpr int kPairs = 8;  // pairs of a pass

// DP: type of the pairs' rows, DY: of dy.  Pairs j0 .. j0 + count of token blockIdx.x,
// j0 = blockIdx.y * count.
template <int DP, int DY>
__global__ __launch_bounds__(1024) void combine_grad_kernel(const CombineGradArgs a, int count) {
    __shared__ float part[16][kPairs];
    const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const size_t row = (size_t)t * a.H;
    for (int b = blockIdx.y * count; b < min(a.k, (int)(blockIdx.y + 1) * count); b += kPairs) {
        const int n = min(kPairs, a.k - b);
        float w[kPairs], sum[kPairs];
        bool here[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const size_t p = (size_t)t * a.k + min(b + j, a.k - 1);
            const int id = a.ids[p];
            // resident iff the slot is in [0, S): the batching kernels' rule
            here[j] = j < n && id >= 0 && id < a.E && (unsigned)a.slot_of_expert[id] < (unsigned)a.S;
            w[j] = a.w[p];
            sum[j] = 0.0f;
        }
        for (int c = threadIdx.x * 8; c < a.H; c += blockDim.x * 8) {
            float dy[8], y[kPairs][8];
            load_vec8<DY>(a.dy, row + c, dy);
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                if (here[j]) load_vec8<DP>(a.y_pairs, ((size_t)t * a.k + b + j) * a.H + c, y[j]);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                if (j >= n) continue;
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (here[j]) sum[j] = fmaf(y[j][i], dy[i], sum[j]);
                    d[i] = here[j] ? w[j] * dy[i] : 0.0f;
                }
                store_vec8<DP>(a.dy_pairs, ((size_t)t * a.k + b + j) * a.H + c, d);
            }
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            sum[j] = wave_sum(sum[j]);
            if (lane == 0) part[wave][j] = sum[j];
        }
        __syncthreads();
        if ((int)threadIdx.x < n) {
            float v = 0.0f;
            for (int u = 0; u < waves; ++u) v += part[u][threadIdx.x];
            a.dw[(size_t)t * a.k + b + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

template <int DP>
static void launch_dy(const CombineGradArgs& a, dim3 grid, int threads, int count, hipStream_t s) {
    if (a.dy_dtype == MOE_F32) combine_grad_kernel<DP, MOE_F32><<<grid, threads, 0, s>>>(a, count);
    else if (a.dy_dtype == MOE_BF16) combine_grad_kernel<DP, MOE_BF16><<<grid, threads, 0, s>>>(a, count);
    else combine_grad_kernel<DP, MOE_F16><<<grid, threads, 0, s>>>(a, count);
}

hipError_t launch_combine_backward(const CombineGradArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const int threads = a.H > 1024 ? 256 : a.H > 512 ? 128 : 64;
    const int count = a.k;
    const dim3 grid(a.T, (a.k + count - 1) / count);
    if (a.pairs_dtype == MOE_F32) launch_dy<MOE_F32>(a, grid, threads, count, s);
    else if (a.pairs_dtype == MOE_BF16) launch_dy<MOE_BF16>(a, grid, threads, count, s);
    else launch_dy<MOE_F16>(a, grid, threads, count, s);
    return hipGetLastError();
}

}  // namespace qmoe
