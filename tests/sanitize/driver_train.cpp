// The argument checks and tables of a training step's operators (csrc/abi_ops.cpp)
// under AddressSanitizer and UndefinedBehaviorSanitizer: sizes at the ends of int
// and of the documented ranges, lists and tables in heap blocks of their exact sizes.
// Every call is refused or has nothing to do, so nothing is enqueued.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <vector>

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
static void* const kOther = reinterpret_cast<void*>(uintptr_t(1) << 21);
static void* const kOdd = reinterpret_cast<void*>((uintptr_t(1) << 20) + 8);
static const int32_t* const kInt = static_cast<const int32_t*>(kBuf);
static float* const kF = static_cast<float*>(kBuf);

static moe_status bias(int S, int N, int K, int R, int k, int act, void* y = kBuf, void* z = nullptr) {
    return moe_expert_gemm_bias(kBuf, MOE_BF16, kBuf, SIZE_MAX & ~size_t(15), S, N, K, kBuf, MOE_F32, nullptr, 0, kInt, R,
                                kInt, k, 0, 0, act, y, MOE_BF16, z, nullptr);
}
static moe_status act(int S, int N, int R, int kind, size_t bytes = SIZE_MAX, void* dz = kOther) {
    return moe_expert_act_backward(kBuf, kBuf, MOE_F32, S, N, kInt, R, kInt, 0, kind, dz, nullptr, kF, kBuf, bytes, nullptr);
}

static void products() {
    for (int e : {INT_MIN, -8, INT_MAX, INT_MAX - 7}) {
        CHECK(bias(e, 64, 128, 8, 2, 0) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(bias(4, e, 128, 8, 2, 0) != MOE_OK);
        CHECK(bias(4, 64, e, 8, 2, 0) != MOE_OK);
        CHECK(bias(4, 64, 128, e, 2, 0) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(bias(4, 64, 128, 8, e, 0) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(bias(4, 64, 128, 8, 2, e) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(act(e, 64, 8, MOE_ACT_GELU) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(act(4, e, 8, MOE_ACT_GELU) != MOE_OK);
        CHECK(act(4, 64, e, MOE_ACT_GELU) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(act(4, 64, 8, e) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(moe_expert_act_backward_workspace_size(e, 64, 8) == 0);
        CHECK(moe_expert_act_backward_workspace_size(4, e, 8) == 0);
        CHECK(moe_expert_act_backward_workspace_size(4, 64, e) == 0);
    }
    CHECK(bias(1024, 1 << 15, 1 << 15, 0, 64, MOE_ACT_SWIGLU) == MOE_OK);  // no rows: nothing to do
    CHECK(bias(4, 64, 128, 8, 2, MOE_ACT_RELU, kBuf, kBuf) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(bias(4, 64, 128, 8, 2, MOE_ACT_RELU, kOdd) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(moe_expert_act_backward_workspace_size(1024, 1 << 20, 1 << 24) > (size_t(1) << 32));
    CHECK(act(4, 64, 8, MOE_ACT_GELU, moe_expert_act_backward_workspace_size(4, 64, 8) - 1) == MOE_ERR_WORKSPACE_TOO_SMALL);
    CHECK(act(4, 64, 8, MOE_ACT_SWIGLU, SIZE_MAX, kBuf) == MOE_ERR_INVALID_ARGUMENT);
}

static moe_status losses(int T, int E, int k, int G, size_t bytes = SIZE_MAX) {
    return moe_balance_loss(kF, kInt, T, E, k, MOE_SCORE_SIGMOID, kInt, G, static_cast<int32_t*>(kBuf), kF, kF, kBuf, bytes,
                            nullptr);
}
static moe_status route(int T, int E, int k, int G, float scale = 1.0f, int out = MOE_BF16) {
    return moe_route_backward(kF, kInt, kF, T, E, k, MOE_SCORE_SOFTMAX, 1, scale, kInt, kF, kInt, G, kOther, out, nullptr);
}
static moe_status combine(int E, int S, int T, int k, int H) {
    return moe_combine_backward(kBuf, MOE_F32, kBuf, MOE_F16, kInt, kF, kInt, E, S, T, k, H, kOther,
                                static_cast<float*>(kOther), nullptr);
}

static void router() {
    for (int e : {INT_MIN, -1, INT_MAX}) {
        CHECK(losses(e, 16, 2, 1) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(losses(8, e, 2, 1) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(losses(8, 16, e, 1) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(losses(8, 16, 2, e) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(route(e, 16, 2, 1) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(route(8, e, 2, 1) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(route(8, 16, e, 1) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(route(8, 16, 2, e) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(route(8, 16, 2, 1, 1.0f, e) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(combine(e, 2, 8, 2, 64) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(combine(16, e, 8, 2, 64) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(combine(16, 2, e, 2, 64) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(combine(16, 2, 8, e, 64) == MOE_ERR_INVALID_ARGUMENT);
        CHECK(combine(16, 2, 8, 2, e) != MOE_OK);
        CHECK(moe_balance_loss_workspace_size(e, 16, 1) == 0);
        CHECK(moe_balance_loss_workspace_size(8, e, 1) == 0);
        CHECK(moe_balance_loss_workspace_size(8, 16, e) == 0);
    }
    CHECK(moe_balance_loss_workspace_size(1 << 24, 1024, 1024) > 0);
    CHECK(losses(1 << 24, 1024, 1, 1024, moe_balance_loss_workspace_size(1 << 24, 1024, 1024) - 1) ==
          MOE_ERR_WORKSPACE_TOO_SMALL);
    CHECK(route(8, 16, 2, 1, NAN) == MOE_ERR_INVALID_ARGUMENT);
    CHECK(route(0, 16, 2, 1) == MOE_OK);
    CHECK(combine(16, 2, 0, 2, 64) == MOE_OK);
}

static void lists() {
    // lists of every length around a launch's, in blocks of their exact sizes
    for (int n : {0, 1, 159, 160, 161, 240, 241, 1000}) {
        std::vector<const void*> at(n);
        std::vector<void*> outs(n);
        std::vector<int64_t> counts(n);
        std::vector<int32_t> types(n);
        for (int i = 0; i < n; ++i) {
            at[i] = kBuf;
            outs[i] = kOther;
            counts[i] = i % 7 ? 1 + int64_t(i) * i : 0;
            types[i] = i % 3;
        }
        std::vector<uint8_t> table(moe_grad_table_size(n));
        CHECK(moe_grad_table(at.data(), counts.data(), types.data(), n, table.data(), table.size()) == MOE_OK);
        CHECK(moe_grad_norm_workspace_size(n) > 0);
        if (n == 0) {
            CHECK(moe_grad_clip(at.data(), counts.data(), types.data(), 0, nullptr, nullptr, nullptr, nullptr, kF, 1.0f, 0.0f,
                                1.0f, nullptr) == MOE_OK);
            continue;
        }
        CHECK(moe_grad_table(at.data(), counts.data(), types.data(), n, table.data(), table.size() - 1) ==
              MOE_ERR_WORKSPACE_TOO_SMALL);
        types[n - 1] = INT_MIN;
        CHECK(moe_grad_norm(at.data(), counts.data(), types.data(), n, nullptr, 0, 1.0f, kF, kBuf, SIZE_MAX, nullptr) ==
              MOE_ERR_INVALID_ARGUMENT);
        types[n - 1] = MOE_F32;
        counts[n - 1] = INT64_MIN;
        CHECK(moe_grad_norm(at.data(), counts.data(), types.data(), n, nullptr, 0, 1.0f, kF, kBuf, SIZE_MAX, nullptr) ==
              MOE_ERR_INVALID_ARGUMENT);
        counts[n - 1] = INT64_MAX;
        CHECK(moe_grad_clip(at.data(), counts.data(), types.data(), n, nullptr, outs.data(), types.data(), nullptr, kF, 1.0f,
                            0.0f, 1.0f, nullptr) == MOE_ERR_INVALID_ARGUMENT);
        counts[n - 1] = int64_t(1) << 40;
        CHECK(moe_grad_table(at.data(), counts.data(), types.data(), n, table.data(), table.size()) == MOE_OK);
        CHECK(moe_grad_clip(at.data(), counts.data(), types.data(), n, nullptr, outs.data(), types.data(), nullptr, kF, NAN,
                            0.0f, 1.0f, nullptr) == MOE_ERR_INVALID_ARGUMENT);
        for (int64_t& c : counts) c = 0;  // nothing to do
        CHECK(moe_grad_clip(at.data(), counts.data(), types.data(), n, kBuf, outs.data(), types.data(), kBuf, kF, 1.0f, 0.0f,
                            1.0f, nullptr) == MOE_OK);
    }
    CHECK(moe_grad_table_size(-1) == 0 && moe_grad_table_size(INT_MAX) == 0 && moe_grad_norm_workspace_size(INT_MIN) == 0);
}

int main() {
    products();
    router();
    lists();
    if (g_failures == 0) std::printf("all passed\n");
    return g_failures != 0;
}
