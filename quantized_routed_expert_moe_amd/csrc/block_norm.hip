// The norm after a block, its gate, the residual sum and the norm before the
// next block in one pass over the rows, and their gradients.
//
// Forward, per row (i1, i2 the reciprocal root mean squares):
//   p = y i1, r = p w_post, x_out = a x + gate r, h = x_out i2 w_pre.
// Backward, with n = x_out i2, dn = dh w_pre and m = mean(dn n):
//   dxo = dx_out + i2 (dn - n m),  dw_pre += dh n,  dx = a dxo,
//   dgate += dxo r,  dr = dxo gate,  dw_post += dr p,  dp = dr w_post,
//   dy = i1 (dp - p mean(dp p)).
// The statistics are recomputed from x and y, so the backward call reads
// what the forward call read plus the two gradients and nothing is saved.
//
// Bound by HBM: every element is read and written once.  TPR threads hold a
// row in registers (VPT chunks of eight elements each, 16-byte accesses for
// the 16-bit types), the channel vectors stay in registers over the rows
// that a workgroup walks, and the next row's loads are issued before this
// row's reductions, so a workgroup's barriers do not leave the memory idle.
// The backward pass needs three row sums that build on each other; the third
// is linear in dxo, so with G = gate w_post p
//   sum(dp p) = sum(dx_out G) + i2 sum(dn G) - i2^2 m sum(x_out G)
// and one barrier serves them all: two reductions a row instead of three.
// Sums over rows (dw_post, dgate, dw_pre) are kept per workgroup in fp32
// registers, written as one partial per workgroup and added in workgroup
// order by a second launch: no atomics, equal bits for equal calls.
#include "device_common.h"
#include "expert_ops.h"

namespace qmoe {

// Eight elements as loaded: one 16-byte word (16-bit types) or two (fp32).
struct Raw8 {
    uint4 a, b;
};
__device__ __forceinline__ Raw8 raw_load(const void* base, int dtype, size_t idx) {
    Raw8 r;
    if (dtype == MOE_F32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + idx);
        r.a = p[0];
        r.b = p[1];
    } else {
        r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + idx);
        r.b = r.a;
    }
    return r;
}
__device__ __forceinline__ void raw_floats(const Raw8& r, int dtype, float* v) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (dtype == MOE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else if (dtype == MOE_BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = half_to_float(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
}
__device__ __forceinline__ void store_any8(void* base, int dtype, size_t idx, const float* v) {
    if (dtype == MOE_F32) store_vec8<MOE_F32>(base, idx, v);
    else if (dtype == MOE_BF16) store_vec8<MOE_BF16>(base, idx, v);
    else store_vec8<MOE_F16>(base, idx, v);
}
__device__ __forceinline__ float load_any(const void* base, int dtype, size_t idx) {
    if (dtype == MOE_F32) return static_cast<const float*>(base)[idx];
    if (dtype == MOE_BF16) return (float)static_cast<const __bf16*>(base)[idx];
    return (float)static_cast<const _Float16*>(base)[idx];
}

// Sums of NV values over the TPR threads of a row, in every thread.  One
// barrier: consecutive calls use alternate halves of `part` (`flip`).
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* part, int& flip) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        float* p = part + flip * (5 * 16);
        flip ^= 1;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i) p[i * 16 + wave] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = row16_sum((lane & 15) < W ? p[i * 16 + (lane & 15)] : 0.0f);
    }
}

// The channel vectors of this thread's chunks: ones where there is none.
template <int VPT>
__device__ __forceinline__ void channel_vector(const void* w, int dtype, int H, int t, int tpr, float (&v)[VPT][8]) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int col = (t + c * tpr) * 8;
        if (w && col < H) {
            raw_floats(raw_load(w, dtype, col), dtype, v[c]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = 1.0f;
        }
    }
}

template <int TPR, int VPT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(const BlockNormArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;  // rows per workgroup
    __shared__ float part[2 * 5 * 16];
    int flip = 0;
    const int t = threadIdx.x % TPR, H = a.H;
    const bool post = a.w_post != nullptr;
    float wpost[VPT][8], gate[VPT][8], wpre[VPT][8];
    channel_vector<VPT>(a.w_post, a.w_dtype, H, t, TPR, wpost);
    channel_vector<VPT>(a.gate_mode == MOE_GATE_CHANNEL ? a.gate : nullptr, a.w_dtype, H, t, TPR, gate);
    channel_vector<VPT>(a.w_pre, a.w_dtype, H, t, TPR, wpre);
#pragma unroll
    for (int c = 0; c < VPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) gate[c][i] *= wpost[c][i];
    const int step = gridDim.x * RPB;
    int row = blockIdx.x * RPB + threadIdx.x / TPR;
    Raw8 rx[VPT], ry[VPT];
    float gt = 1.0f;
    auto fetch = [&](int r) {
        if (r >= a.T) return;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int col = (t + c * TPR) * 8;
            if (col >= H) continue;
            rx[c] = raw_load(a.x, a.dtype, (size_t)r * H + col);
            if (a.y) ry[c] = raw_load(a.y, a.y_dtype, (size_t)r * H + col);
        }
        if (a.gate_mode == MOE_GATE_TOKEN) gt = load_any(a.gate, a.w_dtype, r);
    };
    fetch(row);
    for (; row < a.T; row += step) {
        float x[VPT][8], y[VPT][8];
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const bool in = (t + c * TPR) * 8 < H;
            if (in) raw_floats(rx[c], a.dtype, x[c]);
            if (in && a.y) raw_floats(ry[c], a.y_dtype, y[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[c][i] = in ? x[c][i] * a.res_scale : 0.0f;
                y[c][i] = in && a.y ? y[c][i] : 0.0f;
            }
        }
        const float g = gt;
        fetch(row + step);
        float i1 = g;
        if (post) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < VPT; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[c][i], y[c][i], ss[0]);
            row_sum<TPR, 1>(ss, part, flip);
            i1 *= rsqrtf(ss[0] / (float)H + a.eps);
        }
        float sx[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < VPT; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (a.y) x[c][i] = fmaf(y[c][i] * i1, gate[c][i], x[c][i]);
                sx[0] = fmaf(x[c][i], x[c][i], sx[0]);
            }
        if (a.x_out)
#pragma unroll
            for (int c = 0; c < VPT; ++c) {
                const int col = (t + c * TPR) * 8;
                if (col < H) store_any8(a.x_out, a.dtype, (size_t)row * H + col, x[c]);
            }
        if (a.w_pre) {
            row_sum<TPR, 1>(sx, part, flip);
            const float i2 = rsqrtf(sx[0] / (float)H + a.eps);
#pragma unroll
            for (int c = 0; c < VPT; ++c) {
                const int col = (t + c * TPR) * 8;
                if (col >= H) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * i2 * wpre[c][i];
                store_any8(a.h, a.dtype, (size_t)row * H + col, x[c]);
            }
        }
    }
}

template <int TPR, int VPT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_backward_kernel(const BlockNormArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    __shared__ float part[2 * 5 * 16];
    int flip = 0;
    const int t = threadIdx.x % TPR, H = a.H;
    const bool post = a.w_post != nullptr;
    float wpost[VPT][8], gate[VPT][8], wpre[VPT][8];
    channel_vector<VPT>(a.w_post, a.w_dtype, H, t, TPR, wpost);
    channel_vector<VPT>(a.gate_mode == MOE_GATE_CHANNEL ? a.gate : nullptr, a.w_dtype, H, t, TPR, gate);
    channel_vector<VPT>(a.w_pre, a.w_dtype, H, t, TPR, wpre);
    float s_post[VPT][8] = {}, s_gate[VPT][8] = {}, s_pre[VPT][8] = {};
    const int step = gridDim.x * RPB;
    int row = blockIdx.x * RPB + threadIdx.x / TPR;
    Raw8 rx[VPT], ry[VPT], rdx[VPT], rdh[VPT];
    float gt = 1.0f;
    auto fetch = [&](int r) {
        if (r >= a.T) return;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int col = (t + c * TPR) * 8;
            if (col >= H) continue;
            const size_t at = (size_t)r * H + col;
            rx[c] = raw_load(a.x, a.dtype, at);
            if (a.y) ry[c] = raw_load(a.y, a.y_dtype, at);
            if (a.dx_out) rdx[c] = raw_load(a.dx_out, a.dtype, at);
            if (a.dh) rdh[c] = raw_load(a.dh, a.dtype, at);
        }
        if (a.gate_mode == MOE_GATE_TOKEN) gt = load_any(a.gate, a.w_dtype, r);
    };
    fetch(row);
    for (; row < a.T; row += step) {
        // x becomes x_out, y the normed p, d dx_out, e dn
        float x[VPT][8], y[VPT][8], d[VPT][8], e[VPT][8];
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const bool in = (t + c * TPR) * 8 < H;
            if (in) raw_floats(rx[c], a.dtype, x[c]);
            if (in && a.y) raw_floats(ry[c], a.y_dtype, y[c]);
            if (in && a.dx_out) raw_floats(rdx[c], a.dtype, d[c]);
            if (in && a.dh) raw_floats(rdh[c], a.dtype, e[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[c][i] = in ? x[c][i] : 0.0f;
                y[c][i] = in && a.y ? y[c][i] : 0.0f;
                d[c][i] = in && a.dx_out ? d[c][i] : 0.0f;
                e[c][i] = in && a.dh ? e[c][i] : 0.0f;
            }
        }
        const float g = gt;
        fetch(row + step);
        float i1 = 1.0f;
        if (post) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < VPT; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[c][i], y[c][i], ss[0]);
            row_sum<TPR, 1>(ss, part, flip);
            i1 = rsqrtf(ss[0] / (float)H + a.eps);
        }
        // sums of x_out^2, dn x_out, and of dx_out, dn and x_out with G (the
        // token's gate g left out: sum(dxo G) is then the token gate's gradient)
        float sm[5] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < VPT; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[c][i] *= i1;
                const float G = y[c][i] * wpost[c][i] * gate[c][i];
                const float xo = fmaf(g, G, a.res_scale * x[c][i]);
                const float dn = e[c][i] * wpre[c][i];
                sm[0] = fmaf(xo, xo, sm[0]);
                sm[1] = fmaf(dn, xo, sm[1]);
                sm[2] = fmaf(d[c][i], G, sm[2]);
                sm[3] = fmaf(dn, G, sm[3]);
                sm[4] = fmaf(xo, G, sm[4]);
                x[c][i] = xo;
            }
        row_sum<TPR, 5>(sm, part, flip);
        const float inv = 1.0f / (float)H;
        const float i2 = a.w_pre ? rsqrtf(sm[0] * inv + a.eps) : 0.0f;
        const float m = i2 * sm[1] * inv;                        // mean(dn n)
        const float sG = sm[2] + i2 * (sm[3] - i2 * m * sm[4]);  // sum(dxo G)
        const float mp = g * sG * inv;                           // mean(dp p)
        if (a.gate_mode == MOE_GATE_TOKEN && t == 0) a.dgate[row] = sG;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int col = (t + c * TPR) * 8;
            if (col >= H) continue;
            const size_t at = (size_t)row * H + col;
            float dx[8], dy[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = x[c][i] * i2;
                const float dxo = d[c][i] + i2 * (e[c][i] * wpre[c][i] - n * m);
                s_pre[c][i] = fmaf(e[c][i], n, s_pre[c][i]);
                dx[i] = a.res_scale * dxo;
                const float r = y[c][i] * wpost[c][i];
                s_gate[c][i] = fmaf(dxo, r, s_gate[c][i]);
                const float dr = dxo * gate[c][i] * g;
                s_post[c][i] = fmaf(dr, y[c][i], s_post[c][i]);
                dy[i] = post ? i1 * (dr * wpost[c][i] - y[c][i] * mp) : dr;
            }
            store_any8(a.dx, a.dtype, at, dx);
            if (a.dy) store_any8(a.dy, a.y_dtype, at, dy);
        }
    }
    // the workgroup's partial sums, [workgroup][3][H]; the rows of a workgroup
    // that walks several at a time are added through LDS first, in row order
    float* o = static_cast<float*>(a.ws) + (size_t)blockIdx.x * 3 * H;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int col = (t + c * TPR) * 8;
            if (col >= H) continue;
            store_vec8<MOE_F32>(o, col, s_post[c]);
            store_vec8<MOE_F32>(o + H, col, s_gate[c]);
            store_vec8<MOE_F32>(o + 2 * H, col, s_pre[c]);
        }
    } else {
        __shared__ float buf[RPB * TPR * VPT * 8];
        auto add = [&](float (&v)[VPT][8], float* dst) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < VPT; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) buf[(threadIdx.x / TPR) * TPR * VPT * 8 + (t + c * TPR) * 8 + i] = v[c][i];
            __syncthreads();
            for (int col = threadIdx.x; col < H; col += RPB * TPR) {
                float z = 0.0f;
#pragma unroll
                for (int r = 0; r < RPB; ++r) z += buf[r * TPR * VPT * 8 + col];
                dst[col] = z;
            }
        };
        add(s_post, o);
        add(s_gate, o + H);
        add(s_pre, o + 2 * H);
    }
}

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
#pragma unroll 8
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

// Threads per row and chunks per thread: the fewest threads that hold the
// row in one chunk each up to 1024 threads (8192 columns), two beyond.
struct NormShape {
    int tpr, rpb;
};
static NormShape norm_shape(int H) {
    if (H <= 512) return {64, 4};
    if (H <= 2048) return {256, 1};
    if (H <= 4096) return {512, 1};
    return {1024, 1};
}
static int norm_blocks(int T, int H) {
    const NormShape n = norm_shape(H);
    const int want = (T + n.rpb - 1) / n.rpb, most = 256 * (2048 / (n.tpr * n.rpb));  // two waves a SIMD and more
    return want < most ? want : most;
}

#define NORM_DISPATCH(KERNEL)                                                     \
    if (a.H <= 512) KERNEL<64, 1><<<grid, 256, 0, s>>>(a);                        \
    else if (a.H <= 2048) KERNEL<256, 1><<<grid, 256, 0, s>>>(a);                 \
    else if (a.H <= 4096) KERNEL<512, 1><<<grid, 512, 0, s>>>(a);                 \
    else if (a.H <= 8192) KERNEL<1024, 1><<<grid, 1024, 0, s>>>(a);               \
    else KERNEL<1024, 2><<<grid, 1024, 0, s>>>(a);

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const dim3 grid(norm_blocks(a.T, a.H));
    NORM_DISPATCH(block_norm_kernel)
    return hipGetLastError();
}

size_t block_norm_backward_workspace_bytes(int T, int H) { return (size_t)norm_blocks(T, H) * 3 * H * sizeof(float); }

hipError_t launch_block_norm_backward(const BlockNormArgs& a, hipStream_t s) {
    const dim3 grid(norm_blocks(a.T, a.H));
    if (a.T > 0) {
        NORM_DISPATCH(block_norm_backward_kernel)
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    float* dgate = a.gate_mode == MOE_GATE_CHANNEL ? a.dgate : nullptr;
    if (a.dw_post || dgate || a.dw_pre)
        block_norm_reduce_kernel<<<dim3((a.H + 63) / 64, 3), 1024, 0, s>>>(static_cast<const float*>(a.ws),
                                                                           (int)grid.x, a.H, a.dw_post, dgate,
                                                                           a.dw_pre);
    return hipGetLastError();
}

}  // namespace qmoe
