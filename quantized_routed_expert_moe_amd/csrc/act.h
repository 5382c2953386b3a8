// The activations of the biased products and their derivatives, fp32, eight
// values at a time.  SiLU and the tanh form of GELU are both v sigmoid(a v + b v^3):
// (1 + tanh u) / 2 = sigmoid(2 u).
#pragma once
#include "expert_ops.h"

namespace qmoe {

// v held within +-1e4, where every sigmoid is 0 or 1 to the last bit and v^3 is finite; NaN stays.
__device__ __forceinline__ float act_range(float v) { return v > 1.0e4f ? 1.0e4f : v < -1.0e4f ? -1.0e4f : v; }

constexpr float kGeluA = 1.5957691216057308f;               // 2 sqrt(2 / pi)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

// act(v).
__device__ __forceinline__ float act1(int act, float v) {
    if (act == MOE_ACT_SILU || act == MOE_ACT_GELU_TANH) {
        const float b = act == MOE_ACT_SILU ? 0.0f : kGeluB, a = act == MOE_ACT_SILU ? 1.0f : kGeluA, c = act_range(v);
        return v * sigmoid_f32(c * fmaf(b * c, c, a));
    }
    if (act == MOE_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.7071067811865476f));
    return act == MOE_ACT_RELU && v < 0.0f ? 0.0f : v;
}

// v = act(v): one test of act for the eight.
__device__ __forceinline__ void act8(int act, float* v) {
    if (act == MOE_ACT_NONE) return;
    if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act1(MOE_ACT_GELU, v[i]);
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act1(MOE_ACT_RELU, v[i]);
    } else {
        const float b = act == MOE_ACT_SILU ? 0.0f : kGeluB, a = act == MOE_ACT_SILU ? 1.0f : kGeluA;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = act_range(v[i]);
            v[i] = v[i] * sigmoid_f32(c * fmaf(b * c, c, a));
        }
    }
}

// s = 1 / (1 + e^-u) and q = 1 - s, of one exponential (as in sigmoid_f32).
__device__ __forceinline__ void sigmoid_pair(float u, float& s, float& q) {
    const float t = -1.4426950408889634f * u;
    const float rest = fmaf(-1.4426950408889634f, u, -t) - 1.925963033500e-8f * u;
    const float e0 = __builtin_amdgcn_exp2f(t);
    const float e = e0 > 0.0f && e0 < 3.0e38f ? fmaf(e0, 0.6931471805599453f * rest, e0) : e0;
    s = __builtin_amdgcn_rcpf(1.0f + e);
    q = u < 0.0f ? 1.0f - s : e * s;
}

// Gradients at an infinite z, which stands for a sum beyond its type's range (an fp16 sum past 65504 whose
// activation was finite), are the limits there: the factors that vanish take z held within
// act_range, of which finite z keep their bits.

// dz = d act'(z), h = act(z).
__device__ __forceinline__ void act_grad8(int act, const float* z, const float* d, float* dz, float* h) {
    if (act == MOE_ACT_SILU || act == MOE_ACT_GELU_TANH) {
        const bool silu = act == MOE_ACT_SILU;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = act_range(z[i]);
            const float b = silu ? 0.0f : kGeluB, a = silu ? 1.0f : kGeluA;
            float s, q;
            sigmoid_pair(c * fmaf(b * c, c, a), s, q);
            dz[i] = d[i] * (s * fmaf(c * q, fmaf(3.0f * b * c, c, a), 1.0f));
            h[i] = fmaxf(z[i], -1.0e4f) * s;  // NaN is in s
        }
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = 0.5f * (1.0f + erff(z[i] * 0.7071067811865476f));
            // z e^(-z^2 / 2) / sqrt(2 pi)
            const float t = -0.7213475204444817f * z[i] * z[i];
            const float c = __builtin_amdgcn_fmed3f(z[i], -1.0e4f, 1.0e4f);
            dz[i] = d[i] * fmaf(c, 0.3989422804014327f * __builtin_amdgcn_exp2f(t), p);  // NaN is in p
            h[i] = fmaxf(z[i], -1.0e4f) * p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dz[i] = z[i] > 0.0f ? d[i] : 0.0f;
            h[i] = z[i] < 0.0f ? 0.0f : z[i];
        }
    }
}

// a v, 0 for a = 0 and infinite v.
__device__ __forceinline__ float times_limit(float a, float v) { return a == 0.0f && __builtin_isinf(v) ? 0.0f : a * v; }

// SwiGLU of g and u and its gradient for given d.
__device__ __forceinline__ void swiglu_grad(float g, float u, float d, float& dg, float& du, float& h) {
    const float s = sigmoid_f32(g);
    h = g * s * u;
    dg = d * u * s * (1.0f + g * (1.0f - s));
    du = d * g * s;
}

// The same where g or u may be infinite.
__device__ __forceinline__ void swiglu_grad_limit(float g, float u, float d, float& dg, float& du, float& h) {
    if (!__builtin_isinf(g) && !__builtin_isinf(u)) return swiglu_grad(g, u, d, dg, du, h);
    const float c = act_range(g), s = sigmoid_f32(c), gs = fmaxf(g, -1.0e4f) * s;
    h = __builtin_isinf(gs) ? times_limit(u, gs) : times_limit(gs, u);
    dg = times_limit(d * (s * (1.0f + c * (1.0f - s))), u);
    du = times_limit(d, gs);
}

}  // namespace qmoe
