// C ABI of the expert products, the 4-bit products, the block norms and
// SwiGLU: argument checks and dispatch to the launchers.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "expert_ops.h"

namespace {

moe_status fail(moe_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return qmoe::set_error(st, buf);
}

moe_status launched(hipError_t e, const char* what) {
    if (e == hipSuccess) return MOE_OK;
    return fail(MOE_ERR_HIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool half_type(int t) { return t == MOE_BF16 || t == MOE_F16; }
bool any_type(int t) { return t == MOE_F32 || half_type(t); }

constexpr int kMaxRows = 1 << 24;
constexpr long long kMaxMatrix = 1ll << 30;

// The checks that every product shares.
moe_status check_product(int dtype, int S, int N, int K, const int32_t* slot_offsets, int R, const int32_t* perm_pair,
                         int k, int a_rows, int b_rows, int act) {
    if (!half_type(dtype)) return fail(MOE_ERR_UNSUPPORTED, "dtype = %d is not MOE_BF16 or MOE_F16", dtype);
    if (S < 1 || S > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID_ARGUMENT, "S = %d outside 1..%d", S, MOE_MAX_EXPERTS);
    if (N <= 0 || K <= 0) return fail(MOE_ERR_INVALID_ARGUMENT, "N = %d, K = %d must be positive", N, K);
    if (N % 8 || K % 8) return fail(MOE_ERR_UNSUPPORTED, "N = %d and K = %d must be multiples of 8", N, K);
    if ((long long)N * K > kMaxMatrix) return fail(MOE_ERR_UNSUPPORTED, "N*K = %lld exceeds 2^30", (long long)N * K);
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return fail(MOE_ERR_INVALID_ARGUMENT, "bad act %d", act);
    if (act == MOE_ACT_SWIGLU && N % 16)
        return fail(MOE_ERR_UNSUPPORTED, "MOE_ACT_SWIGLU needs N (%d) a multiple of 16", N);
    if (R < 0 || R > kMaxRows) return fail(MOE_ERR_INVALID_ARGUMENT, "R = %d outside 0..2^24", R);
    if (k < 1 || k > MOE_MAX_TOPK) return fail(MOE_ERR_INVALID_ARGUMENT, "k = %d outside 1..%d", k, MOE_MAX_TOPK);
    for (const int r : {a_rows, b_rows})
        if (r < MOE_ROWS_POSITION || r > MOE_ROWS_TOKEN) return fail(MOE_ERR_INVALID_ARGUMENT, "bad row mode %d", r);
    if (!slot_offsets && S != 1)
        return fail(MOE_ERR_INVALID_ARGUMENT, "slot_offsets is NULL with S = %d (only S = 1 may leave it out)", S);
    if (R > 0 && !perm_pair && (a_rows != MOE_ROWS_POSITION || b_rows != MOE_ROWS_POSITION))
        return fail(MOE_ERR_INVALID_ARGUMENT, "perm_pair is NULL, the row modes need it");
    return MOE_OK;
}

moe_status check_output(int dtype, int out_dtype, const char* name) {
    if (out_dtype != MOE_F32 && out_dtype != dtype)
        return fail(MOE_ERR_UNSUPPORTED, "%s dtype %d is neither the operands' (%d) nor MOE_F32", name, out_dtype,
                    dtype);
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_expert_gemm(const void* x, int dtype, const void* w, size_t w_stride, int S, int N, int K,
                           int transpose, const int32_t* slot_offsets, int R, const int32_t* perm_pair, int k,
                           int x_rows, int y_rows, int act, void* y, int y_dtype, void* stream) {
    moe_status st = check_product(dtype, S, N, K, slot_offsets, R, perm_pair, k, x_rows, y_rows, act);
    if (st != MOE_OK) return st;
    if (transpose != 0 && transpose != 1) return fail(MOE_ERR_INVALID_ARGUMENT, "transpose = %d is not 0 or 1", transpose);
    if (transpose && act) return fail(MOE_ERR_INVALID_ARGUMENT, "MOE_ACT_SWIGLU goes with transpose 0");
    if (y_rows == MOE_ROWS_TOKEN) return fail(MOE_ERR_INVALID_ARGUMENT, "y_rows cannot be MOE_ROWS_TOKEN");
    if ((st = check_output(dtype, y_dtype, "y")) != MOE_OK) return st;
    if (!w || (R > 0 && (!x || !y))) return fail(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (!aligned16(x) || !aligned16(w) || !aligned16(y) || (w_stride & 15u))
        return fail(MOE_ERR_INVALID_ARGUMENT, "x, w, y and w_stride must be 16-byte aligned");
    if (w_stride < (size_t)N * K * 2)
        return fail(MOE_ERR_INVALID_ARGUMENT, "w_stride %zu is smaller than the matrix (%zu bytes)", w_stride,
                    (size_t)N * K * 2);
    const qmoe::ExpertGemmArgs a{x,      w,      w_stride, dtype, N,      K, transpose, qmoe::row_map(slot_offsets, perm_pair, S, R, k),
                                 x_rows, y_rows, act,      y,     y_dtype};
    return launched(qmoe::launch_expert_gemm(a, (hipStream_t)stream), "expert product launch");
}

size_t moe_expert_gemm_wgrad_workspace_size(int S, int N, int K, int R) {
    if (S < 1 || S > MOE_MAX_EXPERTS || N <= 0 || K <= 0 || N % 8 || K % 8 || (long long)N * K > kMaxMatrix || R < 0 ||
        R > kMaxRows)
        return 0;
    return qmoe::expert_wgrad_workspace_bytes(S, N, K, R);
}

moe_status moe_expert_gemm_wgrad(const void* dy, const void* x, int dtype, int S, int N, int K,
                                 const int32_t* slot_offsets, int R, const int32_t* perm_pair, int k, int dy_rows,
                                 int x_rows, void* dw, int dw_dtype, void* ws, size_t ws_bytes, void* stream) {
    moe_status st = check_product(dtype, S, N, K, slot_offsets, R, perm_pair, k, dy_rows, x_rows, MOE_ACT_NONE);
    if (st != MOE_OK) return st;
    if ((st = check_output(dtype, dw_dtype, "dw")) != MOE_OK) return st;
    if (!dw || (R > 0 && (!dy || !x))) return fail(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (!aligned16(dy) || !aligned16(x) || !aligned16(dw))
        return fail(MOE_ERR_INVALID_ARGUMENT, "dy, x and dw must be 16-byte aligned");
    const size_t need = qmoe::expert_wgrad_workspace_bytes(S, N, K, R);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", ws_bytes, need);
    if (need > 0 && (!ws || !aligned16(ws)))
        return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be non-NULL and 16-byte aligned");
    const qmoe::ExpertWgradArgs a{dy, x, dtype, N, K, qmoe::row_map(slot_offsets, perm_pair, S, R, k), dy_rows, x_rows,
                                  dw, dw_dtype, ws};
    return launched(qmoe::launch_expert_wgrad(a, (hipStream_t)stream), "weight gradient launch");
}

moe_status moe_expert_gemv_w4(const void* x, int dtype, const void* q, const void* scales, int scale_dtype,
                              const uint8_t* zeros, int group, int S, int N, int K, const int32_t* slot_offsets,
                              int R, const int32_t* perm_pair, int k, int x_rows, int y_rows, int act, void* y,
                              int y_dtype, void* stream) {
    moe_status st = check_product(dtype, S, N, K, slot_offsets, R, perm_pair, k, x_rows, y_rows, act);
    if (st != MOE_OK) return st;
    if (group != 32 && group != 64 && group != 128)
        return fail(MOE_ERR_UNSUPPORTED, "group = %d is not 32, 64 or 128", group);
    if (K % group) return fail(MOE_ERR_UNSUPPORTED, "K = %d is not a multiple of the group (%d)", K, group);
    if (y_rows == MOE_ROWS_TOKEN) return fail(MOE_ERR_INVALID_ARGUMENT, "y_rows cannot be MOE_ROWS_TOKEN");
    if ((st = check_output(dtype, scale_dtype, "scale")) != MOE_OK) return st;
    if ((st = check_output(dtype, y_dtype, "y")) != MOE_OK) return st;
    if (!q || !scales || (R > 0 && (!x || !y))) return fail(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (!aligned16(x) || !aligned16(q) || !aligned16(scales) || !aligned16(y))
        return fail(MOE_ERR_INVALID_ARGUMENT, "x, q, scales and y must be 16-byte aligned");
    const qmoe::ExpertW4Args a{x, dtype, static_cast<const uint8_t*>(q), scales, scale_dtype, zeros, group, N, K,
                               qmoe::row_map(slot_offsets, perm_pair, S, R, k), x_rows, y_rows, act, y, y_dtype};
    return launched(qmoe::launch_expert_w4(a, (hipStream_t)stream), "4-bit product launch");
}

static moe_status check_norm(const void* x, int dtype, const void* y, int y_dtype, const void* w_post,
                             const void* gate, int gate_mode, const void* w_pre, int w_dtype, int T, int H, float eps,
                             float res_scale) {
    if (T < 0 || T > kMaxRows) return fail(MOE_ERR_INVALID_ARGUMENT, "T = %d outside 0..2^24", T);
    if (H <= 0) return fail(MOE_ERR_INVALID_ARGUMENT, "H = %d must be positive", H);
    if (H % 8 || H > MOE_MAX_NORM_WIDTH)
        return fail(MOE_ERR_UNSUPPORTED, "H = %d is not a multiple of 8 up to %d", H, MOE_MAX_NORM_WIDTH);
    if (!any_type(dtype)) return fail(MOE_ERR_INVALID_ARGUMENT, "bad dtype %d", dtype);
    if (y && !any_type(y_dtype)) return fail(MOE_ERR_INVALID_ARGUMENT, "bad y dtype %d", y_dtype);
    if ((w_post || gate || w_pre) && !any_type(w_dtype)) return fail(MOE_ERR_INVALID_ARGUMENT, "bad w dtype %d", w_dtype);
    if (gate_mode < MOE_GATE_NONE || gate_mode > MOE_GATE_TOKEN)
        return fail(MOE_ERR_INVALID_ARGUMENT, "bad gate mode %d", gate_mode);
    // a [T] gate of no tokens has no storage
    if ((gate_mode != MOE_GATE_NONE) != (gate != nullptr) && !(gate_mode == MOE_GATE_TOKEN && T == 0))
        return fail(MOE_ERR_INVALID_ARGUMENT, "gate and its mode (%d) go together", gate_mode);
    if (T > 0 && !x) return fail(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (T > 0 && !y && (w_post || gate)) return fail(MOE_ERR_INVALID_ARGUMENT, "w_post and gate need y");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    if (!std::isfinite(res_scale)) return fail(MOE_ERR_INVALID_ARGUMENT, "res_scale must be finite");
    if (!aligned16(x) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
        (gate_mode == MOE_GATE_CHANNEL && !aligned16(gate)))
        return fail(MOE_ERR_INVALID_ARGUMENT, "x, y, w_post, gate and w_pre must be 16-byte aligned");
    return MOE_OK;
}

moe_status moe_block_norm(const void* x, int dtype, const void* y, int y_dtype, const void* w_post, const void* gate,
                          int gate_mode, const void* w_pre, int w_dtype, int T, int H, float eps, float res_scale,
                          void* x_out, void* h, void* stream) {
    moe_status st = check_norm(x, dtype, y, y_dtype, w_post, gate, gate_mode, w_pre, w_dtype, T, H, eps, res_scale);
    if (st != MOE_OK) return st;
    if (T > 0 && (w_pre != nullptr) != (h != nullptr)) return fail(MOE_ERR_INVALID_ARGUMENT, "h and w_pre go together");
    if (T > 0 && !x_out && !h) return fail(MOE_ERR_INVALID_ARGUMENT, "neither x_out nor h is given");
    if (!aligned16(x_out) || !aligned16(h)) return fail(MOE_ERR_INVALID_ARGUMENT, "x_out and h must be 16-byte aligned");
    qmoe::BlockNormArgs a{};
    a.x = x; a.dtype = dtype; a.y = y; a.y_dtype = y_dtype; a.w_post = w_post; a.gate = gate; a.gate_mode = gate_mode;
    a.w_pre = w_pre; a.w_dtype = w_dtype; a.T = T; a.H = H; a.eps = eps; a.res_scale = res_scale;
    a.x_out = x_out; a.h = h;
    return launched(qmoe::launch_block_norm(a, (hipStream_t)stream), "block norm launch");
}

size_t moe_block_norm_backward_workspace_size(int T, int H) {
    if (T < 0 || T > kMaxRows || H <= 0 || H % 8 || H > MOE_MAX_NORM_WIDTH) return 0;
    return qmoe::block_norm_backward_workspace_bytes(T, H);
}

moe_status moe_block_norm_backward(const void* x, int dtype, const void* y, int y_dtype, const void* w_post,
                                   const void* gate, int gate_mode, const void* w_pre, int w_dtype, int T, int H,
                                   float eps, float res_scale, const void* dx_out, const void* dh, void* dx,
                                   void* dy, float* dw_post, float* dgate, float* dw_pre, void* ws, size_t ws_bytes,
                                   void* stream) {
    moe_status st = check_norm(x, dtype, y, y_dtype, w_post, gate, gate_mode, w_pre, w_dtype, T, H, eps, res_scale);
    if (st != MOE_OK) return st;
    if (T > 0 && (!dx || (w_pre != nullptr) != (dh != nullptr) || (y != nullptr) != (dy != nullptr)))
        return fail(MOE_ERR_INVALID_ARGUMENT, "dx is required, dh goes with w_pre and dy with y");
    if (T > 0 && !dx_out && !dh) return fail(MOE_ERR_INVALID_ARGUMENT, "neither dx_out nor dh is given");
    if ((w_post != nullptr) != (dw_post != nullptr) || (w_pre != nullptr) != (dw_pre != nullptr) ||
        (gate != nullptr) != (dgate != nullptr))
        return fail(MOE_ERR_INVALID_ARGUMENT, "dw_post, dgate and dw_pre go with w_post, gate and w_pre");
    if (!aligned16(dx_out) || !aligned16(dh) || !aligned16(dx) || !aligned16(dy))
        return fail(MOE_ERR_INVALID_ARGUMENT, "dx_out, dh, dx and dy must be 16-byte aligned");
    const size_t need = qmoe::block_norm_backward_workspace_bytes(T, H);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", ws_bytes, need);
    if (need > 0 && (!ws || !aligned16(ws)))
        return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be non-NULL and 16-byte aligned");
    qmoe::BlockNormArgs a{};
    a.x = x; a.dtype = dtype; a.y = y; a.y_dtype = y_dtype; a.w_post = w_post; a.gate = gate; a.gate_mode = gate_mode;
    a.w_pre = w_pre; a.w_dtype = w_dtype; a.T = T; a.H = H; a.eps = eps; a.res_scale = res_scale;
    a.dx_out = dx_out; a.dh = dh; a.dx = dx; a.dy = dy; a.dw_post = dw_post; a.dgate = dgate; a.dw_pre = dw_pre;
    a.ws = ws;
    return launched(qmoe::launch_block_norm_backward(a, (hipStream_t)stream), "block norm gradient launch");
}

static moe_status check_swiglu(const void* gu, int dtype, int R, int I, const int32_t* slot_offsets, int S) {
    if (!any_type(dtype)) return fail(MOE_ERR_INVALID_ARGUMENT, "bad dtype %d", dtype);
    if (R < 0 || R > kMaxRows) return fail(MOE_ERR_INVALID_ARGUMENT, "R = %d outside 0..2^24", R);
    if (I <= 0) return fail(MOE_ERR_INVALID_ARGUMENT, "I = %d must be positive", I);
    if (I % 8 || I > (1 << 24)) return fail(MOE_ERR_UNSUPPORTED, "I = %d is not a multiple of 8 up to 2^24", I);
    if (S < 0 || S > MOE_MAX_EXPERTS || (S > 0) != (slot_offsets != nullptr))
        return fail(MOE_ERR_INVALID_ARGUMENT, "slot_offsets and S in 1..%d go together (S = %d)", MOE_MAX_EXPERTS, S);
    if (R > 0 && !gu) return fail(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    return MOE_OK;
}

moe_status moe_swiglu(const void* gu, int dtype, int R, int I, const int32_t* slot_offsets, int S, void* h,
                      void* stream) {
    moe_status st = check_swiglu(gu, dtype, R, I, slot_offsets, S);
    if (st != MOE_OK) return st;
    if (R > 0 && !h) return fail(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (!aligned16(gu) || !aligned16(h)) return fail(MOE_ERR_INVALID_ARGUMENT, "gu and h must be 16-byte aligned");
    const qmoe::SwigluArgs a{gu, nullptr, dtype, R, I, slot_offsets, S, nullptr, h};
    return launched(qmoe::launch_swiglu(a, (hipStream_t)stream), "SwiGLU launch");
}

moe_status moe_swiglu_backward(const void* gu, const void* dh, int dtype, int R, int I, const int32_t* slot_offsets,
                               int S, void* dgu, void* h, void* stream) {
    moe_status st = check_swiglu(gu, dtype, R, I, slot_offsets, S);
    if (st != MOE_OK) return st;
    if (R > 0 && (!dh || !dgu)) return fail(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (!aligned16(gu) || !aligned16(dh) || !aligned16(dgu) || !aligned16(h))
        return fail(MOE_ERR_INVALID_ARGUMENT, "gu, dh, dgu and h must be 16-byte aligned");
    const qmoe::SwigluArgs a{gu, dh, dtype, R, I, slot_offsets, S, dgu, h};
    return launched(qmoe::launch_swiglu_backward(a, (hipStream_t)stream), "SwiGLU gradient launch");
}

}  // extern "C"
