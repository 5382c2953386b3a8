// The argument checks of the expert products, the 4-bit products, the block
// norms and SwiGLU (csrc/abi_ops.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer: sizes at the ends of int and of the documented
// ranges, missing and misaligned pointers.  Every call is refused or has
// nothing to do, so nothing is enqueued.  Returns the number of failed checks.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/qmoe.h"

static int g_failures = 0;
#define CHECK(cond)                                                                             \
    do {                                                                                        \
        if (!(cond)) {                                                                          \
            std::fprintf(stderr, "CHECK failed at %s:%d: %s\n", __FILE__, __LINE__, #cond);     \
            ++g_failures;                                                                       \
        }                                                                                       \
    } while (0)

static void* const kBuf = reinterpret_cast<void*>(uintptr_t(1) << 20);  // never dereferenced
static void* const kOdd = reinterpret_cast<void*>((uintptr_t(1) << 20) + 8);
static const int32_t* const kInt = static_cast<const int32_t*>(kBuf);

static moe_status gemm(int S, int N, int K, int R, int k, int dtype = MOE_BF16, size_t stride = SIZE_MAX & ~size_t(15),
                       const void* x = kBuf, void* y = kBuf, int act = 0, int tr = 0, int xr = 0, int yr = 0) {
    return moe_expert_gemm(x, dtype, kBuf, stride, S, N, K, tr, kInt, R, kInt, k, xr, yr, act, y, dtype, nullptr);
}

static void products() {
    const int edges[] = {INT_MIN, -8, 0, INT_MAX, INT_MAX - 7};
    for (int e : edges) {
        CHECK(gemm(4, e, 128, 8, 2) != MOE_OK);
        CHECK(gemm(4, 64, e, 8, 2) != MOE_OK);
        CHECK(gemm(e, 64, 128, 8, 2) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(gemm(4, 64, 128, 8, e) == MOE_ERR_INVALID_ARGUMENT);
        if (e) CHECK(gemm(4, 64, 128, e, 2) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(moe_expert_gemv_w4(kBuf, MOE_F16, kBuf, kBuf, MOE_F32, nullptr, 64, 4, 64, e, kInt, 8, kInt, 2, 0, 0, 0,
                                 kBuf, MOE_F16, nullptr) != MOE_OK);
        CHECK(moe_expert_gemv_w4(kBuf, MOE_F16, kBuf, kBuf, MOE_F32, nullptr, e, 4, 64, 128, kInt, 8, kInt, 2, 0, 0, 0,
                                 kBuf, MOE_F16, nullptr) == MOE_ERR_UNSUPPORTED);
        CHECK(moe_expert_gemm_wgrad(kBuf, kBuf, MOE_BF16, 4, e, 128, kInt, 8, kInt, 2, 0, 0, kBuf, MOE_F32, kBuf, SIZE_MAX,
                                    nullptr) != MOE_OK);
        CHECK(moe_expert_gemm_wgrad_workspace_size(e, 64, 128, 1 << 20) == 0);
        CHECK(moe_expert_gemm_wgrad_workspace_size(1, e, 128, 1 << 20) == 0);
        CHECK(moe_expert_gemm_wgrad_workspace_size(1, 64, e, 1 << 20) == 0);
        if (e) CHECK(moe_expert_gemm_wgrad_workspace_size(1, 64, 128, e) == 0);
    }
    // enums, row modes, pointers, strides
    CHECK(gemm(4, 64, 128, 8, 2, INT_MIN) == MOE_ERR_UNSUPPORTED);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 64 * 128 * 2 - 16) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 64 * 128 * 2 + 8) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 1 << 20, kOdd) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 1 << 20, kBuf, nullptr) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 1 << 20, kBuf, kBuf, 7) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 56, 128, 8, 2, MOE_BF16, 1 << 20, kBuf, kBuf, MOE_ACT_SWIGLU) == MOE_ERR_UNSUPPORTED);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 1 << 20, kBuf, kBuf, MOE_ACT_SWIGLU, 1) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 1 << 20, kBuf, kBuf, 0, INT_MAX) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 1 << 20, kBuf, kBuf, 0, 0, INT_MIN) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 8, 2, MOE_BF16, 1 << 20, kBuf, kBuf, 0, 0, 0, MOE_ROWS_TOKEN) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 64, 128, 0, 2, MOE_BF16, 1 << 20, nullptr, nullptr) == MOE_OK);  // no rows: nothing to do
    // the largest sizes: no overflow on the way to an answer
    CHECK(moe_expert_gemm_wgrad_workspace_size(MOE_MAX_EXPERTS, 1 << 15, 1 << 15, 1 << 24) == 0);
    const size_t parts = moe_expert_gemm_wgrad_workspace_size(1, 256, 256, 1 << 24);
    CHECK(parts > 0 && parts % (256 * 256 * sizeof(float)) == 0);
    CHECK(moe_expert_gemm_wgrad(kBuf, kBuf, MOE_BF16, 1, 256, 256, nullptr, 1 << 24, nullptr, 1, 0, 0, kBuf, MOE_F32, kBuf,
                                parts - 1, nullptr) == MOE_ERR_WORKSPACE_TOO_SMALL);
    CHECK(moe_expert_gemm_wgrad(kBuf, kBuf, MOE_BF16, 1, 256, 256, nullptr, 1 << 24, nullptr, 1, 0, 0, kBuf, MOE_F32, kOdd,
                                parts, nullptr) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(gemm(4, 1 << 16, 1 << 15, 8, 2) == MOE_ERR_UNSUPPORTED);  // N K = 2^31
}

static moe_status norm(int T, int H, float eps = 1e-6f, float a = 1.0f, const void* x = kBuf, const void* gate = kBuf,
                       int mode = MOE_GATE_CHANNEL) {
    return moe_block_norm(x, MOE_BF16, kBuf, MOE_F32, kBuf, gate, mode, kBuf, MOE_F32, T, H, eps, a, kBuf, kBuf, nullptr);
}

static void norms() {
    for (int e : {INT_MIN, -1, INT_MAX, (1 << 24) + 1}) {
        CHECK(norm(e, 64) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(moe_block_norm_backward_workspace_size(e, 64) == 0);
    }
    for (int e : {INT_MIN, -8, 0, 4, 12, MOE_MAX_NORM_WIDTH + 8, INT_MAX, INT_MAX - 7}) {
        CHECK(norm(4, e) != MOE_OK);
        CHECK(moe_block_norm_backward_workspace_size(4, e) == 0);
    }
    CHECK(norm(4, 64, NAN) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, 64, INFINITY) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, 64, 1e-6f, -INFINITY) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, 64, 1e-6f, 1.0f, kOdd) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, 64, 1e-6f, 1.0f, nullptr) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, 64, 1e-6f, 1.0f, kBuf, nullptr) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, 64, 1e-6f, 1.0f, kBuf, kBuf, INT_MAX) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(norm(0, 64) == MOE_OK);  // no rows: nothing to do
    const size_t need = moe_block_norm_backward_workspace_size(1 << 24, MOE_MAX_NORM_WIDTH);
    float* f = static_cast<float*>(kBuf);
    CHECK(need > 0);
    for (size_t have : {size_t(0), need - 1})
        CHECK(moe_block_norm_backward(kBuf, MOE_F32, kBuf, MOE_F16, kBuf, kBuf, MOE_GATE_CHANNEL, kBuf, MOE_F32, 1 << 24,
                                      MOE_MAX_NORM_WIDTH, 1e-6f, 1.0f, kBuf, kBuf, kBuf, kBuf, f, f, f, kBuf, have,
                                      nullptr) == MOE_ERR_WORKSPACE_TOO_SMALL);
    CHECK(moe_block_norm_backward(kBuf, MOE_F32, kBuf, MOE_F16, kBuf, kBuf, MOE_GATE_CHANNEL, kBuf, MOE_F32, 4, 64, 1e-6f,
                                  1.0f, kBuf, kBuf, kBuf, kBuf, f, nullptr, f, kBuf, SIZE_MAX,
                                  nullptr) == MOE_ERR_INVALID_ARGUMENT);
}

static void swiglu() {
    for (int e : {INT_MIN, -1, (1 << 24) + 1, INT_MAX}) {
        CHECK(moe_swiglu(kBuf, MOE_BF16, e, 64, nullptr, 0, kBuf, nullptr) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(moe_swiglu(kBuf, MOE_BF16, 4, e, nullptr, 0, kBuf, nullptr) != MOE_OK);
        CHECK(moe_swiglu(kBuf, e, 4, 64, nullptr, 0, kBuf, nullptr) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(moe_swiglu_backward(kBuf, kBuf, MOE_F32, 4, 64, kInt, e, kBuf, nullptr, nullptr) == MOE_ERR_INVALID_ARGUMENT);
    }
    CHECK(moe_swiglu(kBuf, MOE_BF16, 0, 64, nullptr, 0, nullptr, nullptr) == MOE_OK);
    CHECK(moe_swiglu_backward(kBuf, kBuf, MOE_F32, 4, 64, nullptr, 0, kBuf, kOdd, nullptr) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(std::strlen(moe_last_error()) > 0);
}

int driver_ops() {
    products();
    norms();
    swiglu();
    return g_failures;
}
