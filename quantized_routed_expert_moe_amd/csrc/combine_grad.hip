// The weighted combine's gradients: dy_pairs[p] = w_p dy[t] and dw[p] = <y_pairs[p], dy[t]>.
//
// Bound by HBM: each pair's row is read and one written, a token's row of dy read.
// A workgroup owns eight of a token's pairs: a thread holds eight columns of
// dy and takes them through the pairs, whose loads are in flight together; the
// eight sums are joined in wave order at the end.  Lane j of each wave looks pair j up, so
// that a token's ids, weights and slots are two loads in a row and not sixteen.
// 4096 tokens of 8 pairs of 2048, bf16: 57 us of inputs from HBM (5.0 TB/s), 52 where the
// last-level cache holds a part of them.
#include "train_ops.h"

namespace qmoe {

constexpr int kPairs = 8;  // pairs of a workgroup

// load_vec8 past the caches.
template <int DT>
__device__ __forceinline__ void load_vec8_past(const void* base, size_t idx, float* v) {
    typedef typename DType<DT>::type E;
    constexpr int W = 16 / sizeof(E);
    typedef E vec __attribute__((ext_vector_type(W)));
    const vec* p = reinterpret_cast<const vec*>(static_cast<const E*>(base) + idx);
#pragma unroll
    for (int u = 0; u < 8 / W; ++u) {
        const vec q = __builtin_nontemporal_load(p + u);
#pragma unroll
        for (int i = 0; i < W; ++i) v[u * W + i] = (float)q[i];
    }
}

// DP: type of the pairs' rows, DY: of dy.  PAST: the pairs' rows are read past the caches.
template <int DP, int DY, bool PAST>
__global__ __launch_bounds__(512) void combine_grad_kernel(const CombineGradArgs a) {
    __shared__ float part[8][kPairs];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int passes = (a.k + kPairs - 1) / kPairs;
    for (int unit = blockIdx.x; unit < a.T * passes; unit += gridDim.x) {
        const int t = unit / passes, b = unit % passes * kPairs;
        const size_t row = (size_t)t * a.H, p0 = (size_t)t * a.k;
        const int n = min(kPairs, a.k - b);
        // lane j looks up pair j; all lanes then take it from there
        const int id = a.ids[p0 + b + min(lane, n - 1)];
        const float weight = a.w[p0 + b + min(lane, n - 1)];
        // resident iff the slot is in [0, S): the batching kernels' rule
        const bool resident = id >= 0 && id < a.E && (unsigned)a.slot_of_expert[min(max(id, 0), a.E - 1)] < (unsigned)a.S;
        const uint32_t here = (uint32_t)__ballot(resident && lane < n);
        float w[kPairs], sum[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            w[j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
            sum[j] = 0.0f;
        }
        for (int c = threadIdx.x * 8; c < a.H; c += blockDim.x * 8) {
            float dy[8], y[kPairs][8];
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                if (here >> j & 1) {
                    if (PAST) load_vec8_past<DP>(a.y_pairs, (p0 + b + j) * a.H + c, y[j]);
                    else load_vec8<DP>(a.y_pairs, (p0 + b + j) * a.H + c, y[j]);
                }
            load_vec8<DY>(a.dy, row + c, dy);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                if (j >= n) continue;
                float d[8] = {};
                if (here >> j & 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sum[j] = fmaf(y[j][i], dy[i], sum[j]);
                        d[i] = w[j] * dy[i];
                    }
                }
                store_vec8<DP>(a.dy_pairs, (p0 + b + j) * a.H + c, d);
            }
        }
        float mine = 0.0f;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            if (j >= n) continue;  // a sum over the lanes costs as much as a row of 512
            const float v = wave_sum(sum[j]);
            if (lane == j) mine = v;
        }
        if (waves == 1) {
            if (lane < n) a.dw[p0 + b + lane] = mine;
            continue;
        }
        if (lane < kPairs) part[wave][lane] = mine;
        __syncthreads();
        if ((int)threadIdx.x < n) {
            float v = 0.0f;
            for (int u = 0; u < waves; ++u) v += part[u][threadIdx.x];
            a.dw[p0 + b + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

template <int DP, bool PAST>
static void launch_dy(const CombineGradArgs& a, int threads, hipStream_t s) {
    // up to 2^20 workgroups, which then take several units: a launch's threads stay below 2^32
    const int units = a.T * ((a.k + kPairs - 1) / kPairs);
    const dim3 grid(units < (1 << 20) ? units : 1 << 20);
    if (a.dy_dtype == MOE_F32) combine_grad_kernel<DP, MOE_F32, PAST><<<grid, threads, 0, s>>>(a);
    else if (a.dy_dtype == MOE_BF16) combine_grad_kernel<DP, MOE_BF16, PAST><<<grid, threads, 0, s>>>(a);
    else combine_grad_kernel<DP, MOE_F16, PAST><<<grid, threads, 0, s>>>(a);
}

template <bool PAST>
static void launch_pairs(const CombineGradArgs& a, int threads, hipStream_t s) {
    if (a.pairs_dtype == MOE_F32) launch_dy<MOE_F32, PAST>(a, threads, s);
    else if (a.pairs_dtype == MOE_BF16) launch_dy<MOE_BF16, PAST>(a, threads, s);
    else launch_dy<MOE_F16, PAST>(a, threads, s);
}

hipError_t launch_combine_backward(const CombineGradArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    // A wave for each 512 columns, up to eight: 4096 tokens of 8 x 2048 by 1, 2 and 4 waves 64, 60
    // and 55 us; 333 of 6 x 7168 by 4, 8 and 14 20.4, 14.4 and 15.9.
    const int waves = (a.H + 511) / 512, threads = 64 * (waves < 8 ? waves : 8);
    // The pairs' rows are not read again: past the caches where the last level holds less than
    // them and their gradient (4096 tokens of 8 x 2048: 55.2 us through, 52.3 past), through
    // where it may hold them from before (333 of 6 x 7168: 14.4 and 20.4).
    const size_t bytes = 2 * (size_t)a.T * a.k * a.H * (a.pairs_dtype == MOE_F32 ? 4 : 2);
    if (bytes >= (256u << 20)) launch_pairs<true>(a, threads, s);
    else launch_pairs<false>(a, threads, s);
    return hipGetLastError();
}

}  // namespace qmoe
