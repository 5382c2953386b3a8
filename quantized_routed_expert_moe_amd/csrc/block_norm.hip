// Launches of the block norms (block_norm.h) and the sum of their partial
// channel gradients.
#include "block_norm.h"

namespace qmoe {

// Column sums of the partials: 64 columns x 16 part groups per workgroup,
// each group's parts in order, then the groups in order.
__global__ __launch_bounds__(1024) void block_norm_reduce_kernel(const float* __restrict__ ws, int parts, int H,
                                                                 float* d0, float* d1, float* d2) {
    float* dst = blockIdx.y == 0 ? d0 : blockIdx.y == 1 ? d1 : d2;
    if (!dst) return;
    __shared__ float buf[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (col < H) {
        const float* p = ws + (size_t)blockIdx.y * H + col;
#pragma unroll 16
        for (int i = grp; i < parts; i += 16) v += p[(size_t)i * 3 * H];
    }
    buf[grp][lane] = v;
    __syncthreads();
    if (grp == 0 && col < H) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += buf[i][lane];
        dst[col] = v;
    }
}

// Rows a workgroup takes at a time (the kernels' choice by H in block_norm.h).
static int rows_at_a_time(int H) {
    return H <= 128 ? norm_rows(16) : H <= 256 ? norm_rows(32) : H <= 512 ? norm_rows(64) : 1;
}
// Workgroups: as many as the CUs hold (2048 threads each), so that each walks
// its rows with the channel vectors in registers.
static int norm_blocks(int T, int H) {
    const int threads = H <= 2048 ? 256 : H <= 4096 ? 512 : 1024, rows = rows_at_a_time(H);
    const int want = (T + rows - 1) / rows, most = 256 * (2048 / threads);
    return want < most ? want : most;
}
// The backward pass holds three times the registers and writes a partial sum
// for each workgroup: 512 threads a CU.  (1024: 4099 rows of 2048 take 37.6
// instead of 31.6 us, 20000 rows of 512 36.2 instead of 31.9 us.)
static int norm_backward_blocks(int T, int H) {
    const int threads = H <= 2048 ? 256 : 512, rows = rows_at_a_time(H);
    const int want = (T + rows - 1) / rows, most = 256 * (512 / threads);
    return want < most ? want : most;
}

static hipError_t launch(const BlockNormArgs& a, int backward, int blocks, hipStream_t s) {
    if (a.dtype == MOE_F32) norm_launch_f32(a, backward, dim3(blocks), s);
    else if (a.dtype == MOE_BF16) norm_launch_bf16(a, backward, dim3(blocks), s);
    else norm_launch_f16(a, backward, dim3(blocks), s);
    return hipGetLastError();
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s) {
    return a.T == 0 ? hipSuccess : launch(a, 0, norm_blocks(a.T, a.H), s);
}

size_t block_norm_backward_workspace_bytes(int T, int H) {
    return (size_t)norm_backward_blocks(T, H) * 3 * H * sizeof(float);
}

hipError_t launch_block_norm_backward(const BlockNormArgs& a, hipStream_t s) {
    const int blocks = norm_backward_blocks(a.T, a.H);
    if (a.T > 0) {
        const hipError_t e = launch(a, 1, blocks, s);
        if (e != hipSuccess) return e;
    }
    float* dgate = a.gate_mode == MOE_GATE_CHANNEL ? a.dgate : nullptr;
    if (a.dw_post || dgate || a.dw_pre)
        block_norm_reduce_kernel<<<dim3((a.H + 63) / 64, 3), 1024, 0, s>>>(static_cast<const float*>(a.ws), blocks, a.H,
                                                                           a.dw_post, dgate, a.dw_pre);
    return hipGetLastError();
}

}  // namespace qmoe
