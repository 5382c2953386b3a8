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
// row in registers as loaded (VPT chunks of eight elements each, 16-byte
// accesses for the 16-bit types; each use converts again, which is cheaper
// than twice the registers), the channel vectors stay in registers over the
// rows that a workgroup walks, and the next row's loads are issued before
// this row's reductions, so its barriers do not leave the memory idle.
// The backward pass needs three row sums that build on each other; the third
// is linear in dxo, so with G = gate w_post p
//   sum(dp p) = sum(dx_out G) + i2 sum(dn G) - i2^2 m sum(x_out G)
// and one barrier serves them all: two reductions a row instead of three.
// Sums over rows (dw_post, dgate, dw_pre) are kept per workgroup in fp32
// registers, written as one partial per workgroup and added in workgroup
// order by a second launch: no atomics, equal bits for equal calls.
// Measured: 4099 rows of 2048 (fp16, token gate) 14.6 us, 4.6 TB/s; gradient of
// 8192 rows of 7168 (bf16) 143 us, 5.0 TB/s; 4 rows of 7168 3.8 us.
#pragma once
#include "device_common.h"
#include "expert_ops.h"

namespace qmoe {

// Eight elements as loaded.
template <int DT> struct Raw8 {
    uint4 w[DT == MOE_F32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ void raw_load(Raw8<DT>& r, const void* base, size_t idx) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + idx * (DT == MOE_F32 ? 4 : 2));
    r.w[0] = p[0];
    if constexpr (DT == MOE_F32) r.w[1] = p[1];
}
template <int DT>
__device__ __forceinline__ void raw_floats(const Raw8<DT>& r, float* v) {
    if constexpr (DT == MOE_F32) {
        const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (DT == MOE_BF16) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
            else v[i] = half_to_float(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
        }
    }
}
// Makes the compiler convert again behind this point instead of keeping the floats.
template <int DT>
__device__ __forceinline__ void raw_opaque(Raw8<DT>& r) {
#pragma unroll
    for (int i = 0; i < (DT == MOE_F32 ? 2 : 1); ++i)
        asm("" : "+v"(r.w[i].x), "+v"(r.w[i].y), "+v"(r.w[i].z), "+v"(r.w[i].w));
}
__device__ __forceinline__ float load_any(const void* base, int dtype, size_t idx) {
    if (dtype == MOE_F32) return static_cast<const float*>(base)[idx];
    if (dtype == MOE_BF16) return (float)static_cast<const __bf16*>(base)[idx];
    return (float)static_cast<const _Float16*>(base)[idx];
}
__device__ __forceinline__ void load_any8(const void* base, int dtype, size_t idx, float* v) {
    if (dtype == MOE_F32) load_vec8<MOE_F32>(base, idx, v);
    else if (dtype == MOE_BF16) load_vec8<MOE_BF16>(base, idx, v);
    else load_vec8<MOE_F16>(base, idx, v);
}

// Sums of NV values over the TPR threads of a row, in every thread.  One
// barrier: consecutive calls use alternate halves of `part` (`flip`).
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* part, int& flip) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = TPR == 16 ? row16_sum(v[i]) : TPR == 32 ? half_wave_sum(v[i]) : wave_sum(v[i]);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        float* p = part + flip * (5 * 16);
        flip ^= 1;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i) p[i * 16 + wave] = v[i];
        // LDS only: the next row's loads stay in flight across the barrier
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = row16_sum((lane & 15) < W ? p[i * 16 + (lane & 15)] : 0.0f);
    }
}

// A channel vector at one chunk: ones where there is none.
__device__ __forceinline__ void channel(const void* w, int dtype, int H, int col, float* v) {
    if (w && col < H) {
        load_any8(w, dtype, col, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    }
}

constexpr int norm_rows(int tpr) { return tpr < 256 ? 256 / tpr : 1; }  // rows of a workgroup at a time

template <int XT, int YT, int TPR, int VPT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(const BlockNormArgs a) {
    constexpr int RPB = norm_rows(TPR);
    __shared__ float part[2 * 5 * 16];
    int flip = 0;
    const int t = threadIdx.x % TPR, H = a.H;
    const bool post = a.w_post != nullptr;
    const void* cgate = a.gate_mode == MOE_GATE_CHANNEL ? a.gate : nullptr;
    const int step = gridDim.x * RPB;
    int row = blockIdx.x * RPB + threadIdx.x / TPR;
    Raw8<XT> rx[VPT];
    Raw8<YT> ry[VPT];
    float gt = 1.0f;
    auto fetch = [&](int r) {
        if (r >= a.T) return;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int col = (t + c * TPR) * 8;
            if (col >= H) continue;
            raw_load<XT>(rx[c], a.x, (size_t)r * H + col);
            if (a.y) raw_load<YT>(ry[c], a.y, (size_t)r * H + col);
        }
        if (a.gate_mode == MOE_GATE_TOKEN) gt = load_any(a.gate, a.w_dtype, r);
    };
    fetch(row);
    float gate[VPT][8], wpre[VPT][8];  // gate holds gate * w_post
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int col = (t + c * TPR) * 8;
        float wpost[8];
        channel(a.w_post, a.w_dtype, H, col, wpost);
        channel(cgate, a.w_dtype, H, col, gate[c]);
        channel(a.w_pre, a.w_dtype, H, col, wpre[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) gate[c][i] *= wpost[i];
    }
    const float inv = 1.0f / (float)H;
    for (; row < a.T; row += step) {
        float x[VPT][8], y[VPT][8];
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const bool in = (t + c * TPR) * 8 < H;
            if (in) raw_floats<XT>(rx[c], x[c]);
            if (in && a.y) raw_floats<YT>(ry[c], y[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[c][i] = in ? x[c][i] * a.res_scale : 0.0f;
                y[c][i] = in && a.y ? y[c][i] : 0.0f;
            }
        }
        float i1 = gt;
        fetch(row + step);
        if (post) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < VPT; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[c][i], y[c][i], ss[0]);
            row_sum<TPR, 1>(ss, part, flip);
            i1 *= rsqrtf(ss[0] * inv + a.eps);
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
                if (col < H) store_vec8<XT>(a.x_out, (size_t)row * H + col, x[c]);
            }
        if (a.w_pre) {
            row_sum<TPR, 1>(sx, part, flip);
            const float i2 = rsqrtf(sx[0] * inv + a.eps);
#pragma unroll
            for (int c = 0; c < VPT; ++c) {
                const int col = (t + c * TPR) * 8;
                if (col >= H) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * i2 * wpre[c][i];
                store_vec8<XT>(a.h, (size_t)row * H + col, x[c]);
            }
        }
    }
}

// LEAN: a row is not loaded ahead and the channel vectors are read again for
// every row (four chunks a thread leave no registers for them).
template <int XT, int YT, int TPR, int VPT, bool LEAN>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_backward_kernel(const BlockNormArgs a) {
    constexpr int RPB = norm_rows(TPR);
    __shared__ float part[2 * 5 * 16];
    int flip = 0;
    const int t = threadIdx.x % TPR, H = a.H;
    const bool post = a.w_post != nullptr;
    const void* cgate = a.gate_mode == MOE_GATE_CHANNEL ? a.gate : nullptr;
    const int step = gridDim.x * RPB;
    int row = blockIdx.x * RPB + threadIdx.x / TPR;
    struct Row {
        Raw8<XT> x[VPT], d[VPT], e[VPT];
        Raw8<YT> y[VPT];
        float g;
    } now = {}, next = {};
    now.g = next.g = 1.0f;
    auto fetch = [&](Row& v, int r) {
        if (r >= a.T) return;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int col = (t + c * TPR) * 8;
            if (col >= H) continue;
            const size_t at = (size_t)r * H + col;
            raw_load<XT>(v.x[c], a.x, at);
            if (a.y) raw_load<YT>(v.y[c], a.y, at);
            if (a.dx_out) raw_load<XT>(v.d[c], a.dx_out, at);
            if (a.dh) raw_load<XT>(v.e[c], a.dh, at);
        }
        if (a.gate_mode == MOE_GATE_TOKEN) v.g = load_any(a.gate, a.w_dtype, r);
    };
    if (!LEAN) fetch(next, row);
    float kpost[LEAN ? 1 : VPT][8], kgate[LEAN ? 1 : VPT][8], kpre[LEAN ? 1 : VPT][8];
    if (!LEAN)
#pragma unroll
        for (int c = 0; c < (LEAN ? 1 : VPT); ++c) {
            const int col = (t + c * TPR) * 8;
            channel(a.w_post, a.w_dtype, H, col, kpost[c]);
            channel(cgate, a.w_dtype, H, col, kgate[c]);
            channel(a.w_pre, a.w_dtype, H, col, kpre[c]);
        }
    float s_post[VPT][8] = {}, s_gate[VPT][8] = {}, s_pre[VPT][8] = {};
    const float inv = 1.0f / (float)H;
    for (; row < a.T; row += step) {
        if (LEAN) {
            fetch(now, row);
        } else {
            now = next;
            fetch(next, row + step);
        }
        // Chunks behind H and absent tensors were never loaded: they are zeros.
        float i1 = 1.0f;
        if (post) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < VPT; ++c) {
                float y[8];
                raw_floats<YT>(now.y[c], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[i], y[i], ss[0]);
                raw_opaque<YT>(now.y[c]);
            }
            row_sum<TPR, 1>(ss, part, flip);
            i1 = rsqrtf(ss[0] * inv + a.eps);
        }
        // sums of x_out^2, dn x_out, and of dx_out, dn and x_out with G (the
        // token's gate left out: sum(dxo G) is then the token gate's gradient)
        float sm[5] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        auto vectors = [&](int c, float* wpost, float* gate, float* wpre) {
            const int col = (t + c * TPR) * 8;
            if (LEAN) {
                channel(a.w_post, a.w_dtype, H, col, wpost);
                channel(cgate, a.w_dtype, H, col, gate);
                channel(a.w_pre, a.w_dtype, H, col, wpre);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    wpost[i] = kpost[LEAN ? 0 : c][i];
                    gate[i] = kgate[LEAN ? 0 : c][i];
                    wpre[i] = kpre[LEAN ? 0 : c][i];
                }
            }
        };
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            float x[8], y[8], d[8], e[8], wpost[8], gate[8], wpre[8];
            raw_floats<XT>(now.x[c], x);
            raw_floats<YT>(now.y[c], y);
            raw_floats<XT>(now.d[c], d);
            raw_floats<XT>(now.e[c], e);
            vectors(c, wpost, gate, wpre);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float G = y[i] * i1 * wpost[i] * gate[i];
                const float xo = fmaf(now.g, G, a.res_scale * x[i]);
                const float dn = e[i] * wpre[i];
                sm[0] = fmaf(xo, xo, sm[0]);
                sm[1] = fmaf(dn, xo, sm[1]);
                sm[2] = fmaf(d[i], G, sm[2]);
                sm[3] = fmaf(dn, G, sm[3]);
                sm[4] = fmaf(xo, G, sm[4]);
            }
            raw_opaque<XT>(now.x[c]);
            raw_opaque<YT>(now.y[c]);
            raw_opaque<XT>(now.d[c]);
            raw_opaque<XT>(now.e[c]);
        }
        row_sum<TPR, 5>(sm, part, flip);
        // Without a next norm no gradient holds x_out: its terms are left out, not
        // taken times zero (x_out may be infinite, its sums may overflow).
        const bool pre = a.w_pre != nullptr;
        const float i2 = pre ? rsqrtf(sm[0] * inv + a.eps) : 0.0f;
        const float m = pre ? i2 * sm[1] * inv : 0.0f;                               // mean(dn n)
        const float sG = pre ? sm[2] + i2 * (sm[3] - i2 * m * sm[4]) : sm[2];        // sum(dxo G)
        const float mp = now.g * sG * inv;                                           // mean(dp p)
        if (a.gate_mode == MOE_GATE_TOKEN && t == 0) a.dgate[row] = sG;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int col = (t + c * TPR) * 8;
            if (col >= H) continue;
            const size_t at = (size_t)row * H + col;
            float x[8], y[8], d[8], e[8], wpost[8], gate[8], wpre[8];
            raw_floats<XT>(now.x[c], x);
            raw_floats<YT>(now.y[c], y);
            raw_floats<XT>(now.d[c], d);
            raw_floats<XT>(now.e[c], e);
            vectors(c, wpost, gate, wpre);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = y[i] * i1, r = p * wpost[i];
                const float n = pre ? fmaf(now.g, r * gate[i], a.res_scale * x[i]) * i2 : 0.0f;
                const float dxo = fmaf(i2, fmaf(e[i], wpre[i], -n * m), d[i]);
                const float dr = dxo * gate[i] * now.g;
                s_pre[c][i] = fmaf(e[i], n, s_pre[c][i]);
                s_gate[c][i] = fmaf(dxo, r, s_gate[c][i]);
                s_post[c][i] = fmaf(dr, p, s_post[c][i]);
                x[i] = a.res_scale * dxo;
                y[i] = post ? i1 * fmaf(dr, wpost[i], -p * mp) : dr;
            }
            store_vec8<XT>(a.dx, at, x);
            if (a.dy) store_vec8<YT>(a.dy, at, y);
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

template <int XT, int YT>
static void norm_forward(const BlockNormArgs& a, dim3 grid, hipStream_t s) {
    if (a.H <= 128) block_norm_kernel<XT, YT, 16, 1><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 256) block_norm_kernel<XT, YT, 32, 1><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 512) block_norm_kernel<XT, YT, 64, 1><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 2048) block_norm_kernel<XT, YT, 256, 1><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 4096) block_norm_kernel<XT, YT, 512, 1><<<grid, 512, 0, s>>>(a);
    else if (a.H <= 8192) block_norm_kernel<XT, YT, 1024, 1><<<grid, 1024, 0, s>>>(a);
    else block_norm_kernel<XT, YT, 1024, 2><<<grid, 1024, 0, s>>>(a);
}
template <int XT, int YT>
static void norm_backward(const BlockNormArgs& a, dim3 grid, hipStream_t s) {
    if (a.H <= 128) block_norm_backward_kernel<XT, YT, 16, 1, false><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 256) block_norm_backward_kernel<XT, YT, 32, 1, false><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 512) block_norm_backward_kernel<XT, YT, 64, 1, false><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 2048) block_norm_backward_kernel<XT, YT, 256, 1, false><<<grid, 256, 0, s>>>(a);
    else if (a.H <= 4096) block_norm_backward_kernel<XT, YT, 512, 1, false><<<grid, 512, 0, s>>>(a);
    else if (a.H <= 8192) block_norm_backward_kernel<XT, YT, 512, 2, false><<<grid, 512, 0, s>>>(a);
    else block_norm_backward_kernel<XT, YT, 512, 4, true><<<grid, 512, 0, s>>>(a);
}
template <int XT>
static void norm_launch_type(const BlockNormArgs& a, int backward, dim3 grid, hipStream_t s) {
    const int yt = a.y ? a.y_dtype : XT;
    if (yt == MOE_F32) backward ? norm_backward<XT, MOE_F32>(a, grid, s) : norm_forward<XT, MOE_F32>(a, grid, s);
    else if (yt == MOE_BF16) backward ? norm_backward<XT, MOE_BF16>(a, grid, s) : norm_forward<XT, MOE_BF16>(a, grid, s);
    else backward ? norm_backward<XT, MOE_F16>(a, grid, s) : norm_forward<XT, MOE_F16>(a, grid, s);
}

void norm_launch_f32(const BlockNormArgs& a, int backward, dim3 grid, hipStream_t s);
void norm_launch_bf16(const BlockNormArgs& a, int backward, dim3 grid, hipStream_t s);
void norm_launch_f16(const BlockNormArgs& a, int backward, dim3 grid, hipStream_t s);

}  // namespace qmoe
