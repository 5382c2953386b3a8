// Matrix products grouped by expert over ragged batches and the weight
// gradient: which kernel takes a call.
#include <algorithm>

#include "expert_stream.h"
#include "expert_tile.h"

namespace qmoe {

// Slots that can own a position.
static int possible_slots(const RowMap& m) { return !m.offsets ? 1 : m.S < m.R ? m.S : m.R; }

hipError_t launch_expert_gemm(const ExpertGemmArgs& a, hipStream_t s) {
    if (a.rows.R == 0) return hipSuccess;
    const int slots = possible_slots(a.rows);
    // Few rows a slot: the weights' stream bounds the call.  Up to how many the
    // streaming kernel is the faster one depends on the tiles that the other
    // would have.  Times are us streamed / tiled, bf16.  Few tiles leave CUs idle:
    //   64 (8192 x 2048, one slot)   16 / 20 at 32 rows, 21 / 20 at 48, 25 / 20 at 64
    //   128 (8 slots of 2048 x 2048) 18 / 28 at 12, 23 / 29 at 32, 37 / 28 at 48
    //   256 (16 of 2048 x 2048)      30 / 32 at 2, 31 / 32 at 8, 35 / 32 at 12
    // Enough of them read the weights as fast, and only their start and store count,
    // which a long contraction hides (64 slots of 2048 x K, 1024 tiles):
    //   K = 1024  46 / 50 at 2, 47 / 50 at 8, 52 / 50 at 12
    //   K = 1536  70 / 78 at 2, 76 / 79 at 8, 83 / 80 at 12
    //   K = 2048  98 / 91 at 2, 103 / 93 at 8
    //   K = 4096  228 / 173 at 2
    // With SwiGLU the steps lie lower: 128 slots of 1536 x 2048 156 / 137 at 2.  One rule
    // for all leaves up to a quarter at 13 to 32 rows of 128 tiles and at long K.
    const long long tiles = (long long)slots * ((a.N + 127) / 128);
    const int few = tiles <= 64 ? 48 : tiles <= 128 || a.K < 1536 ? 12 : 2;
    if (!a.transpose && a.rows.R <= (long long)few * slots) {
        const StreamArgs t{a.x, a.w, a.w_stride, nullptr, nullptr, 0, 0, a.N, a.K, a.rows, a.x_rows, a.y_rows, a.y,
                           a.y_dtype == MOE_F32};
        return a.dtype == MOE_BF16 ? launch_stream_bf16(t, 0, a.act, s) : launch_stream_f16(t, 0, a.act, s);
    }
    TileArgs t{};
    t.q = a.x; t.p = a.w; t.p_stride = a.w_stride; t.N = a.N; t.K = a.K; t.rows = a.rows; t.q_rows = a.x_rows;
    t.y_rows = a.y_rows; t.y = a.y; t.y_f32 = a.y_dtype == MOE_F32; t.splits = 1;
    // 256 x 256 tiles once they fill the 256 CUs, else 128 x 128.
    const long long cols = a.transpose ? a.K : a.N;
    const int big = (a.rows.R / 256 + slots) * ((cols + 255) / 256) >= 256;
    const int mode = a.transpose ? kDataGrad : kForward;
    return a.dtype == MOE_BF16 ? launch_tile_bf16(t, mode, a.act, big, s) : launch_tile_f16(t, mode, a.act, big, s);
}

// Parts that a slot's rows are split into where the output has too few tiles
// for the CUs: 128 x 128 tiles and parts of 512 rows and more, up to 16.
static int wgrad_splits(int S, int N, int K, int R) {
    const long long tiles = (long long)S * ((N + 127) / 128) * ((K + 127) / 128);
    const long long most = std::min<long long>(16, R / S / 512);
    return (int)std::max<long long>(1, std::min<long long>(most, 512 / tiles));
}

size_t expert_wgrad_workspace_bytes(int S, int N, int K, int R) {
    const int splits = wgrad_splits(S, N, K, R);
    return splits > 1 ? (size_t)splits * S * N * K * sizeof(float) : 0;
}

// dw = the sum of the parts, in part order.
template <int DT>
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ parts, int splits, size_t n, void* dw) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    float v[8];
    load_vec8<MOE_F32>(parts, i, v);
    for (int p = 1; p < splits; ++p) {
        float u[8];
        load_vec8<MOE_F32>(parts, (size_t)p * n + i, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += u[e];
    }
    store_vec8<DT>(dw, i, v);
}

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t s) {
    TileArgs t{};
    t.q = a.dy; t.p = a.x; t.N = a.N; t.K = a.K; t.rows = a.rows; t.q_rows = a.dy_rows; t.p_rows = a.x_rows;
    t.splits = wgrad_splits(a.rows.S, a.N, a.K, a.rows.R);
    t.y = t.splits > 1 ? a.ws : a.dw;
    t.y_f32 = t.splits > 1 || a.dw_dtype == MOE_F32;
    // 256 x 256 tiles where they fill the CUs and the products count as much as the
    // store of dw, else 128 x 128, of which more share a CU.  128 slots of 1408 x 2048,
    // us by large and by small tiles, fp32: 264 and 224 at a mean of half a row, 254 and
    // 231 at 32, 346 and 335 at 128, 378 and 512 at 256; bf16: 130 and 120 at 4, 118 and
    // 134 at 16.  Rows that end inside a line of 128 bytes cost large tiles more: 60 of
    // 1072 x 1448, fp32: 186 and 83 at 16, 178 and 170 at 256; bf16 93 and 97 at 192.
    const size_t row = (size_t)a.K * (a.dw_dtype == MOE_F32 ? 4 : 2);
    const int few = row % 128 ? 192 : a.dw_dtype == MOE_F32 ? 32 : 8;
    const long long tiles = (long long)a.rows.S * ((a.N + 255) / 256) * ((a.K + 255) / 256);
    const int big = t.splits == 1 && tiles >= 256 && a.rows.R > (long long)few * a.rows.S;
    const hipError_t e = a.dtype == MOE_BF16 ? launch_tile_bf16(t, kWeightGrad, 0, big, s)
                                             : launch_tile_f16(t, kWeightGrad, 0, big, s);
    if (e != hipSuccess || t.splits == 1) return e;
    const size_t n = (size_t)a.rows.S * a.N * a.K;
    const dim3 grid((uint32_t)((n / 8 + 255) / 256));
    const float* parts = static_cast<const float*>(a.ws);
    if (a.dw_dtype == MOE_F32) wgrad_join_kernel<MOE_F32><<<grid, 256, 0, s>>>(parts, t.splits, n, a.dw);
    else if (a.dw_dtype == MOE_BF16) wgrad_join_kernel<MOE_BF16><<<grid, 256, 0, s>>>(parts, t.splits, n, a.dw);
    else wgrad_join_kernel<MOE_F16><<<grid, 256, 0, s>>>(parts, t.splits, n, a.dw);
    return hipGetLastError();
}

}  // namespace qmoe
