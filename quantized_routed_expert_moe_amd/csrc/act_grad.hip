// The activations' gradients with the biases' sums: dz = dy act'(z) and, for
// each slot, the sum of its rows of dz.
//
// Bound by HBM (dy, z, dz and h once each).  A workgroup owns up to `per` rows of one
// slot and a run of columns; a thread takes eight columns through every rl-th
// row and holds their sums, which the workgroup joins and stores as one part; a
// second launch adds a slot's parts in order.  No atomics.
#include "act.h"
#include "train_ops.h"

namespace qmoe {

// Rows of a workgroup: about 2048 workgroups.
static int part_rows(int S, int N, int R) {
    int per = 16;
    const long long chunks = (N + 255) / 256;
    while (per < 4096 && (long long)R / per * chunks > 2048) per *= 2;
    return per;
}
static long long part_count(int S, int R, int per) { return (long long)R / per + (S < R ? S : R); }

size_t act_grad_workspace_bytes(int S, int N, int R) {
    return 4 * 1028 + (size_t)part_count(S, R, part_rows(S, N, R)) * N * sizeof(float);
}

// ACT 0: dz is dy, only the sums are wanted; 1: SwiGLU; 2: another activation.
// A row has 2^cl_shift lanes of eight features.
template <int DT, int KIND>
__global__ __launch_bounds__(256) void act_grad_kernel(const ActGradArgs a, int per, int cl_shift) {
    constexpr int W = KIND == 1 ? 16 : 8;  // sums of a thread
    __shared__ float red[256 * W];
    const int cl = 1 << cl_shift, rl = 256 >> cl_shift, N = a.N, I = KIND == 1 ? N / 2 : N;
    int slot, q0, nq;
    int32_t* prefix = a.dbias && blockIdx.x == 0 && blockIdx.y == 0 ? static_cast<int32_t*>(a.ws) : nullptr;
    if (!find_part<256>(a.rows, per, blockIdx.x, prefix, slot, q0, nq)) return;
    const int lane = threadIdx.x & (cl - 1), c = (blockIdx.y * cl + lane) * 8;
    const bool in = c < I;
    float sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    if (in)
        for (int r = threadIdx.x >> cl_shift; r < nq; r += rl) {
            const size_t row = row_of(a.rows, a.how, q0 + r);
            float d[8], z[8], u[8], dz[8], du[8], h[8];
            load_vec8<DT>(a.dy, row * I + c, d);
            if (KIND) load_vec8<DT>(a.z, row * N + c, z);
            if (KIND == 1) load_vec8<DT>(a.z, row * N + I + c, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (KIND == 1) {
                    const float s = sigmoid_f32(z[i]);
                    h[i] = z[i] * s * u[i];
                    dz[i] = d[i] * u[i] * s * (1.0f + z[i] * (1.0f - s));
                    du[i] = d[i] * z[i] * s;
                    sum[8 % W + i] += du[i];
                } else {
                    dz[i] = d[i];
                }
            }
            if (KIND == 2) act_grad8(a.act, z, d, dz, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += dz[i];
            if (KIND) {
                store_vec8<DT>(a.dz, row * N + c, dz);
                if (KIND == 1) store_vec8<DT>(a.dz, row * N + I + c, du);
                if (a.h) store_vec8<DT>(a.h, row * I + c, h);
            }
        }
    if (!a.dbias) return;
    const int wide = cl * 8;  // features of the workgroup
#pragma unroll
    for (int i = 0; i < W; ++i)
        red[(threadIdx.x >> cl_shift) * wide * (W / 8) + (i / 8) * wide + lane * 8 + i % 8] = sum[i];
    __syncthreads();
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + 4 * 1028) + (size_t)blockIdx.x * N;
    for (int o = threadIdx.x; o < wide * (W / 8); o += 256) {
        const int feature = blockIdx.y * wide + o % wide;
        if (feature >= I) continue;
        float v = 0.0f;
        for (int r = 0; r < rl; ++r) v += red[r * wide * (W / 8) + o];
        part[o / wide * I + feature] = v;
    }
}

// dbias_s = the sum of the slot's parts: 64 columns by four lanes, whose sums are added in order.
__global__ __launch_bounds__(256) void act_grad_join_kernel(const void* ws, int parts, int N, float* dbias) {
    __shared__ float red[256];
    const int32_t* prefix = static_cast<const int32_t*>(ws);
    const int s = blockIdx.x, n = blockIdx.y * 64 + (threadIdx.x & 63), lane = threadIdx.x >> 6;
    const int from = prefix[s], to = min(prefix[s + 1], parts);
    const float* part = reinterpret_cast<const float*>(static_cast<const uint8_t*>(ws) + 4 * 1028);
    float v = 0.0f;
    if (n < N)
        for (int p = from + lane; p < to; p += 4) v += part[(size_t)p * N + n];
    red[threadIdx.x] = v;
    __syncthreads();
    if (lane == 0 && n < N) dbias[(size_t)s * N + n] = ((red[threadIdx.x] + red[threadIdx.x + 64]) + red[threadIdx.x + 128]) + red[threadIdx.x + 192];
}

// No positions: every sum is zero.
__global__ __launch_bounds__(256) void zero_kernel(float* p, size_t n) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

template <int DT>
static void launch_kind(const ActGradArgs& a, dim3 grid, int per, int shift, hipStream_t s) {
    if (a.act == MOE_ACT_NONE) act_grad_kernel<DT, 0><<<grid, 256, 0, s>>>(a, per, shift);
    else if (a.act == MOE_ACT_SWIGLU) act_grad_kernel<DT, 1><<<grid, 256, 0, s>>>(a, per, shift);
    else act_grad_kernel<DT, 2><<<grid, 256, 0, s>>>(a, per, shift);
}

hipError_t launch_act_grad(const ActGradArgs& a, hipStream_t s) {
    const int S = a.rows.S, R = a.rows.R, N = a.N, I = a.act == MOE_ACT_SWIGLU ? N / 2 : N;
    if (R == 0) {
        if (!a.dbias) return hipSuccess;
        const size_t n = (size_t)S * N;
        zero_kernel<<<dim3((uint32_t)((n + 255) / 256)), 256, 0, s>>>(a.dbias, n);
        return hipGetLastError();
    }
    const int per = part_rows(S, N, R);
    int shift = 5;
    while (shift > 0 && (8 << (shift - 1)) >= I) --shift;
    const long long parts = part_count(S, R, per), chunks = (I + (8 << shift) - 1) / (8 << shift);
    if (parts > 0x7FFFFFFFll || chunks > 65535) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)parts, (uint32_t)chunks);
    if (a.dtype == MOE_F32) launch_kind<MOE_F32>(a, grid, per, shift, s);
    else if (a.dtype == MOE_BF16) launch_kind<MOE_BF16>(a, grid, per, shift, s);
    else launch_kind<MOE_F16>(a, grid, per, shift, s);
    if (a.dbias) act_grad_join_kernel<<<dim3(S, (N + 63) / 64), 256, 0, s>>>(a.ws, (int)parts, N, a.dbias);
    return hipGetLastError();
}

}  // namespace qmoe
