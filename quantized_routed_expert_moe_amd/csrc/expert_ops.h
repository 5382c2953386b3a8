// Internal declarations of the expert products, the 4-bit products, the
// block norms and SwiGLU, and the device helpers they share.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qmoe.h"

namespace qmoe {

// Sets the calling thread's error text (abi.cpp).
moe_status set_error(moe_status st, const char* text);

// The rows of a grouped product: batch position -> row of an operand.
struct RowMap {
    const int32_t* offsets;  // [S + 1], or NULL: slot 0 owns all R positions
    const int32_t* perm;     // [R], or NULL
    int S, R, k;
    // p / k = p inv_k >> 30 for p < 2^24 and k <= 64, with inv_k = 2^30 / k
    // rounded up: the excess p (k - 1) / (k 2^30) stays below 1 / k.
    uint32_t inv_k;
};
inline RowMap row_map(const int32_t* offsets, const int32_t* perm, int S, int R, int k) {
    return {offsets, perm, S, R, k, ((1u << 30) + k - 1) / k};
}

// What a biased product does behind its sums: z = sum + bias, y = act(z) + residual.
struct Epilogue {
    const void* bias;  // [S, N], or NULL
    int bias_f32;
    const void* residual;  // as y, or NULL
    int res_f32;
    void* z;  // [R, N], or NULL
    int act;
};

struct ExpertGemmArgs {
    const void* x;
    const void* w;
    size_t w_stride;  // bytes
    int dtype, N, K, transpose;
    RowMap rows;
    int x_rows, y_rows, act;
    void* y;
    int y_dtype;
    const Epilogue* epilogue;  // NULL: none but SwiGLU
};
hipError_t launch_expert_gemm(const ExpertGemmArgs& a, hipStream_t s);

struct ExpertWgradArgs {
    const void* dy;
    const void* x;
    int dtype, N, K;
    RowMap rows;
    int dy_rows, x_rows;
    void* dw;
    int dw_dtype;
    void* ws;
};
size_t expert_wgrad_workspace_bytes(int S, int N, int K, int R);
hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t s);

struct ExpertW4Args {
    const void* x;
    int dtype;
    const uint8_t* q;
    const void* scales;
    int scale_dtype;
    const uint8_t* zeros;
    int group, N, K;
    RowMap rows;
    int x_rows, y_rows, act;
    void* y;
    int y_dtype;
};
hipError_t launch_expert_w4(const ExpertW4Args& a, hipStream_t s);

struct BlockNormArgs {
    const void* x;
    int dtype;
    const void* y;
    int y_dtype;
    const void* w_post;
    const void* gate;
    int gate_mode;
    const void* w_pre;
    int w_dtype, T, H;
    float eps, res_scale;
    void* x_out;  // forward
    void* h;
    const void* dx_out;  // backward
    const void* dh;
    void* dx;
    void* dy;
    float* dw_post;
    float* dgate;
    float* dw_pre;
    void* ws;
};
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s);
size_t block_norm_backward_workspace_bytes(int T, int H);
hipError_t launch_block_norm_backward(const BlockNormArgs& a, hipStream_t s);

struct SwigluArgs {
    const void* gu;
    const void* dh;
    int dtype, R, I;
    const int32_t* offsets;
    int S;
    void* dgu;
    void* h;
};
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s);
hipError_t launch_swiglu_backward(const SwigluArgs& a, hipStream_t s);

#ifdef __HIPCC__

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Device type of a moe_dtype.
template <int DT> struct DType;
template <> struct DType<MOE_F32> { typedef float type; };
template <> struct DType<MOE_BF16> { typedef __bf16 type; };
template <> struct DType<MOE_F16> { typedef _Float16 type; };

// Eight consecutive elements as fp32 (16-byte aligned), and back with one
// rounding each (round to nearest even; the conversions carry NaN).
template <int DT>
__device__ __forceinline__ void load_vec8(const void* base, size_t idx, float* v) {
    if constexpr (DT == MOE_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else if constexpr (DT == MOE_BF16) {
        const bf16x8 u = *reinterpret_cast<const bf16x8*>(static_cast<const __bf16*>(base) + idx);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)u[i];
    } else {
        const f16x8 u = *reinterpret_cast<const f16x8*>(static_cast<const _Float16*>(base) + idx);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)u[i];
    }
}
template <int DT>
__device__ __forceinline__ void store_vec8(void* base, size_t idx, const float* v) {
    if constexpr (DT == MOE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + idx);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (DT == MOE_BF16) {
        bf16x8 u;
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = (__bf16)v[i];
        *reinterpret_cast<bf16x8*>(static_cast<__bf16*>(base) + idx) = u;
    } else {
        f16x8 u;
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = (_Float16)v[i];
        *reinterpret_cast<f16x8*>(static_cast<_Float16*>(base) + idx) = u;
    }
}

// 1 / (1 + e^-z).  log2(e) z is split into its rounded value and the rest,
// so the error stays at a few 2^-24 for large |z| too (the hardware exp2 of
// the rounded product alone loses |z| 2^-24); v_rcp_f32 is within 1 ulp.
__device__ __forceinline__ float sigmoid_f32(float z) {
    const float t = -1.4426950408889634f * z;
    const float rest = fmaf(-1.4426950408889634f, z, -t) - 1.925963033500e-8f * z;
    const float e = __builtin_amdgcn_exp2f(t);
    // e 2^rest = e (1 + ln2 rest); an infinite or zero e (rest may be NaN) stays what it is
    const float ec = fmaf(e, 0.6931471805599453f * rest, e);
    return __builtin_amdgcn_rcpf(1.0f + (e > 0.0f && e < 3.0e38f ? ec : e));
}

// First position and count of slot s, clamped to the R positions.
__device__ __forceinline__ int2 slot_range(const RowMap& m, int s) {
    if (!m.offsets) return make_int2(0, m.R);
    const int a = min(max(m.offsets[s], 0), m.R), b = min(max(m.offsets[s + 1], 0), m.R);
    return make_int2(a, max(b - a, 0));
}

// Token of pair p.
__device__ __forceinline__ int token_of(const RowMap& m, int p) { return (int)__umulhi((uint32_t)p << 2, m.inv_k); }

// Row of an operand for batch position q (q in [0, R)); the pair is clamped
// to [0, R), so a bad permutation reads or writes inside the operand.
__device__ __forceinline__ int row_of(const RowMap& m, int how, int q) {
    if (how == MOE_ROWS_POSITION) return q;
    const int p = min(max(m.perm[q], 0), m.R - 1);
    return how == MOE_ROWS_PAIR ? p : token_of(m, p);
}

// row_of in two parts: the pair (or position) as loaded, and its row.
__device__ __forceinline__ int pair_of(const RowMap& m, int how, int q) {
    return how == MOE_ROWS_POSITION ? q : m.perm[q];
}
__device__ __forceinline__ int row_of_pair(const RowMap& m, int how, int p) {
    p = min(max(p, 0), m.R - 1);
    return how == MOE_ROWS_TOKEN ? token_of(m, p) : p;
}

#endif  // __HIPCC__

}  // namespace qmoe
