// Internal declarations of the operators of a training step: the activations'
// and biases' gradients, the router's losses and gradient, the combine's
// gradient, the gradient norm and clipping; and the device helpers they share.
#pragma once
#include "device_common.h"
#include "expert_ops.h"

namespace qmoe {

struct ActGradArgs {
    const void* dy;
    const void* z;
    int dtype, N;
    RowMap rows;
    int how, act;
    void* dz;
    void* h;
    float* dbias;
    void* ws;
};
size_t act_grad_workspace_bytes(int S, int N, int R);
hipError_t launch_act_grad(const ActGradArgs& a, hipStream_t s);

struct RouterArgs {
    const float* logits;
    const int32_t* ids;
    int T, E, k, score;
    RowMap seqs;  // offsets of the G sequences
    // losses
    int32_t* counts_out;
    float* probs;
    float* losses;
    void* ws;
    // gradient
    const float* dw;
    int renormalize;
    float scale;
    const int32_t* counts;
    const float* dlosses;
    void* dlogits;
    int out_dtype;
};
size_t balance_loss_workspace_bytes(int T, int E, int G);
hipError_t launch_balance_loss(const RouterArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouterArgs& a, hipStream_t s);

struct CombineGradArgs {
    const void* dy;
    int dy_dtype;
    const void* y_pairs;
    int pairs_dtype;
    const int32_t* ids;
    const float* w;
    const int32_t* slot_of_expert;
    int E, S, T, k, H;
    void* dy_pairs;
    float* dw;
};
hipError_t launch_combine_backward(const CombineGradArgs& a, hipStream_t s);

struct GradListArgs {
    const void* const* grads;
    const int64_t* counts;
    const int32_t* dtypes;
    void* const* outs;  // clipping; NULL: in place
    const int32_t* out_dtypes;
    int n, kind;
    float scale, max_norm, eps;
    float* total;
    void* ws;
    const void* table;  // on the device, or NULL
    const void* out_table;
};
size_t grad_table_bytes(int n);
void fill_grad_table(const void* const* at, const int64_t* counts, const int32_t* dtypes, int n, void* table);
size_t grad_norm_workspace_bytes(int n);
hipError_t launch_grad_norm(const GradListArgs& a, hipStream_t s);
hipError_t launch_grad_clip(const GradListArgs& a, hipStream_t s);

#ifdef __HIPCC__

// e^x.  log2(e) x is split into its rounded value and the rest, as in
// sigmoid_f32; 0 below the range, -inf included.
__device__ __forceinline__ float exp_f32(float x) {
    const float t = 1.4426950408889634f * x;
    const float rest = fmaf(1.4426950408889634f, x, -t) + 1.925963033500e-8f * x;
    const float e = __builtin_amdgcn_exp2f(t);
    return e > 0.0f && e < 3.0e38f ? fmaf(e, 0.6931471805599453f * rest, e) : e;
}

// e^x for x <= 0 (or NaN).
__device__ __forceinline__ float exp_down(float x) {
    x = x < -104.0f ? -104.0f : x;  // e^-104 is 0 in fp32
    const float t = 1.4426950408889634f * x;
    const float rest = fmaf(1.925963033500e-8f, x, fmaf(1.4426950408889634f, x, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, 0.6931471805599453f * rest, e);
}

// max(v, the value DPP_CTRL moves into this lane); lanes that get none keep v.  NaN is passed over.
template <int DPP_CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), DPP_CTRL, ROW_MASK,
                                                               0xF, false)));
}

// Largest value and sum over each group of L = 16 or 64 lanes, in all of them.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    v = dpp_max<0x140>(v);
    if (L == 16) return v;
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    return L == 16 ? row16_sum(v) : wave_sum(v);
}

// Value of lane J of each group of L lanes (J < L).
template <int L, int J>
__device__ __forceinline__ int lanes_get(int v) {
    if constexpr (L == 16) return __builtin_amdgcn_update_dpp(0, v, 0x150 + J, 0xF, 0xF, false);  // row_newbcast
    else return __builtin_amdgcn_readlane(v, J);
}

// Sum over the four groups of 16 lanes, lane by lane, in all of them.
__device__ __forceinline__ float sum_of_rows(float v) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Part `index` of the slots' rows, cut into parts of `per` rows each, slots in
// order: its slot, first position and rows.  Found by one scan over the slots
// (S <= 1024) of the whole workgroup; false if there are fewer parts.  prefix, if
// not NULL, receives the parts before each slot, [S + 1].
template <int THREADS>
__device__ __forceinline__ bool find_part(const RowMap& m, int per, int index, int32_t* prefix, int& slot, int& q0,
                                          int& nq) {
    __shared__ int wsum[THREADS / 64], found[3];
    constexpr int PER = 1024 / THREADS;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    if (m.S == 1) {
        const int2 r = slot_range(m, 0);
        slot = 0;
        q0 = r.x + index * per;
        nq = min(per, r.y - index * per);
        if (prefix && t < 2) prefix[t] = t * ((r.y + per - 1) / per);
        return nq > 0;
    }
    int2 r[PER];
    int parts = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int s = t * PER + j;
        r[j] = s < m.S ? slot_range(m, s) : make_int2(0, 0);
        parts += (r[j].y + per - 1) / per;
    }
    int sum = parts;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(sum, o, 64);
        if (lane >= o) sum += x;
    }
    if (lane == 63) wsum[wave] = sum;
    if (t == 0) found[0] = -1;
    __syncthreads();
    sum -= parts;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w)
        if (w < wave) sum += wsum[w];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int s = t * PER + j, n = (r[j].y + per - 1) / per, at = index - sum;
        if (prefix && s <= m.S) prefix[s] = sum;
        if (at >= 0 && at < n) {
            found[0] = s;
            found[1] = r[j].x + at * per;
            found[2] = min(per, r[j].y - at * per);
        }
        sum += n;
    }
    if (prefix && m.S == 1024 && t == THREADS - 1) prefix[m.S] = sum;
    __syncthreads();
    slot = __builtin_amdgcn_readfirstlane(found[0]);
    q0 = __builtin_amdgcn_readfirstlane(found[1]);
    nq = __builtin_amdgcn_readfirstlane(found[2]);
    return slot >= 0;
}

#endif  // __HIPCC__

}  // namespace qmoe
