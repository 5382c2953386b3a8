// The activations' gradients with the biases' sums: dz = dy act'(z) and, for
// each slot, the sum of its rows of dz.
//
// Bound by HBM (dy, z, dz and h once each).  A workgroup owns up to `per` rows of one
// slot and a run of columns; a thread takes eight columns through every rl-th
// row and holds their sums, which the workgroup joins and stores as one part; a
// second launch adds a slot's parts in order.  No atomics.  32768 rows of 768 of 128 slots (SwiGLU,
// h again, bf16): 67 us of inputs from HBM (4.5 TB/s) and 4 us for the sums.  A wave's test for infinite
// halves is 1 % of it (66.4 and 67.2 us).
#include <algorithm>

#include "act.h"
#include "train_ops.h"

namespace qmoe {

constexpr int kRows = 2;  // rows that a thread has in flight

// Lanes of eight features that a row of n of them has, as a power of two up to 32.
static int lane_shift(int n) {
    int shift = 5;
    while (shift > 0 && (8 << (shift - 1)) >= n) --shift;
    return shift;
}

// Rows of a workgroup: two for each thread, and more for 16384 elements a workgroup while that
// leaves 512 of them (32768 rows of 768, SwiGLU: 82 us with 1024 workgroups, 67 with 2048, 66 with 4096 and
// 8192; 1001 rows of 2048 12 us in parts of 16 rows, 15 in 64), and for at most 1024 parts, which the
// second launch adds (the sums alone of 16384 rows of 128: 23 us with 1024 parts and four columns a
// lane for 256 of them, 10 so; 2^20 of 64: 96 with 4096 parts, 26 so, 5.2 TB/s).
static int least_rows(int N) { return 2 * (256 >> lane_shift(N)); }
static long long most_groups(int N, int R) {
    const long long work = (long long)R * N / 16384;
    return work < 512 ? 512 : work < 4096 ? work : 4096;
}
static int part_rows(int N, int R) {
    const long long chunks = (N + 255) / 256, most = most_groups(N, R);
    int per = least_rows(N);
    while (R / per > 1024 || R / per * chunks > most) per *= 2;
    return per;
}
static long long part_count(int S, int R, int per) { return (long long)R / per + (S < R ? S : R); }

// The parts' number falls where their rows double, the need does not: it is what part_rows
// allows.  With p = R / per, p N is at most R / least_rows N, 1024 N and 256 p chunks <= 256 most
// (chunks is N / 256 rounded up), each of which grows with R and N.
size_t act_grad_workspace_bytes(int S, int N, int R) {
    const long long held = std::min({(long long)(R / least_rows(N)) * N, 1024ll * N, 256 * most_groups(N, R)});
    return 4 * 1028 + (size_t)(held + (long long)std::min(S, R) * N) * sizeof(float);
}

// Eight elements in their own type: 16-bit ones stay packed until they are used.
template <int DT> using Vec8 __attribute__((ext_vector_type(8))) = typename DType<DT>::type;
template <int DT>
__device__ __forceinline__ Vec8<DT> load_as(const void* base, size_t at) {
    typedef Vec8<DT> vec __attribute__((aligned(16)));
    return *reinterpret_cast<const vec*>(static_cast<const typename DType<DT>::type*>(base) + at);
}
// acc, made NaN if an element is infinite or NaN (0 v is NaN then).
template <int DT>
__device__ __forceinline__ float not_finite(Vec8<DT> v, float acc) {
    typedef typename DType<DT>::type pair __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        if constexpr (DT == MOE_F32) acc = fmaf(0.0f, v[i], fmaf(0.0f, v[i + 1], acc));
        else if constexpr (DT == MOE_BF16) acc = __builtin_amdgcn_fdot2_f32_bf16(pair{v[i], v[i + 1]}, pair{0, 0}, acc, false);
        else acc = __builtin_amdgcn_fdot2(pair{v[i], v[i + 1]}, pair{0, 0}, acc, false);
    }
    return acc;
}

template <int DT>
__device__ __forceinline__ float load_one(const void* p, size_t at) {
    return (float)static_cast<const typename DType<DT>::type*>(p)[at];
}
template <int DT>
__device__ __forceinline__ void store_one(void* p, size_t at, float v) {
    typedef typename DType<DT>::type E;
    static_cast<E*>(p)[at] = (E)v;
}

// KIND 0: dz is dy, only the sums are wanted; 1: SwiGLU; 2: another activation.
// A row has 2^cl_shift lanes of eight features.
template <int DT, int KIND>
__global__ __launch_bounds__(256) void act_grad_kernel(const ActGradArgs a, int per, int cl_shift) {
    constexpr int W = KIND == 1 ? 16 : 8;  // sums of a thread
    __shared__ float red[256 * W];
    const int cl = 1 << cl_shift, rl = 256 >> cl_shift, N = a.N, I = KIND == 1 ? N / 2 : N;
    int slot, q0, nq;
    int32_t* prefix = a.dbias && blockIdx.x == 0 && blockIdx.y == 0 ? static_cast<int32_t*>(a.ws) : nullptr;
    if (!find_part<256>(a.rows, per, blockIdx.y, prefix, slot, q0, nq)) return;
    const int lane = threadIdx.x & (cl - 1), c = (blockIdx.x * cl + lane) * 8;
    const bool in = c < I;
    float sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    if (in)
        for (int r0 = threadIdx.x >> cl_shift; r0 < nq; r0 += kRows * rl) {
            size_t row[kRows];
            Vec8<DT> zr[kRows], ur[kRows], dr[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int r = r0 + j * rl;
                if (r >= nq) continue;
                row[j] = row_of(a.rows, a.how, q0 + r);
                if (KIND) zr[j] = load_as<DT>(a.z, row[j] * N + c);
                if (KIND == 1) ur[j] = load_as<DT>(a.z, row[j] * N + I + c);
                dr[j] = load_as<DT>(a.dy, row[j] * I + c);
            }
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                if (r0 + j * rl >= nq) continue;
                if (KIND == 1 && __any(not_finite<DT>(zr[j], not_finite<DT>(ur[j], 0.0f)) != 0.0f)) {
                    // one element at a time, loaded again: registers are what the loop is short of
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        float dg, du, h;
                        swiglu_grad_limit(load_one<DT>(a.z, row[j] * N + c + i), load_one<DT>(a.z, row[j] * N + I + c + i),
                                          load_one<DT>(a.dy, row[j] * I + c + i), dg, du, h);
                        store_one<DT>(a.dz, row[j] * N + c + i, dg);
                        store_one<DT>(a.dz, row[j] * N + I + c + i, du);
                        if (a.h) store_one<DT>(a.h, row[j] * I + c + i, h);
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            sum[t] += t == i ? dg : 0.0f;
                            sum[8 % W + t] += t == i ? du : 0.0f;
                        }
                    }
                    continue;
                }
                float z[8], u[8], d[8], dz[8], du[8], h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (KIND) z[i] = (float)zr[j][i];
                    if (KIND == 1) u[i] = (float)ur[j][i];
                    d[i] = (float)dr[j][i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (KIND == 1) swiglu_grad(z[i], u[i], d[i], dz[i], du[i], h[i]);
                    if (KIND == 0) dz[i] = d[i];
                }
                if (KIND == 2) act_grad8(a.act, z, d, dz, h);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)  // the same sums wherever the compiler puts the products
                    sum[i] += dz[i];
                    if (KIND == 1) sum[8 % W + i] += du[i];
                }
                if (KIND) {
                    store_vec8<DT>(a.dz, row[j] * N + c, dz);
                    if (KIND == 1) store_vec8<DT>(a.dz, row[j] * N + I + c, du);
                    if (a.h) store_vec8<DT>(a.h, row[j] * I + c, h);
                }
            }
        }
    if (!a.dbias) return;
    const int wide = cl * 8;  // features of the workgroup
#pragma unroll
    for (int i = 0; i < W; ++i)
        red[(threadIdx.x >> cl_shift) * wide * (W / 8) + (i / 8) * wide + lane * 8 + i % 8] = sum[i];
    __syncthreads();
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + 4 * 1028) + (size_t)blockIdx.y * N;
    for (int o = threadIdx.x; o < wide * (W / 8); o += 256) {
        const int feature = blockIdx.x * wide + o % wide;
        if (feature >= I) continue;
        float v = 0.0f;
        for (int r = 0; r < rl; ++r) v += red[r * wide * (W / 8) + o];
        part[o / wide * I + feature] = v;
    }
}

// dbias_s = the sum of the slot's parts: up to 256 columns, four a thread, by as many lanes as there
// are threads left, whose sums are added as a tree.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void act_grad_join_kernel(const void* ws, int parts, int N, int cl_shift, float* dbias) {
    __shared__ f32x4 red[THREADS];
    const int32_t* prefix = static_cast<const int32_t*>(ws);
    const int cl = 1 << cl_shift, lanes = THREADS >> cl_shift, lane = threadIdx.x >> cl_shift;
    const int s = blockIdx.x, n = (blockIdx.y * cl + (threadIdx.x & (cl - 1))) * 4;
    const int from = prefix[s], to = min(prefix[s + 1], parts);
    const float* part = reinterpret_cast<const float*>(static_cast<const uint8_t*>(ws) + 4 * 1028);
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n < N)
        for (int p = from + lane; p < to; p += lanes) v += *reinterpret_cast<const f32x4*>(part + (size_t)p * N + n);
    red[threadIdx.x] = v;
    for (int half = lanes / 2; half > 0; half /= 2) {
        __syncthreads();
        if (lane < half) red[threadIdx.x] = v += red[threadIdx.x + half * cl];
    }
    if (lane == 0 && n < N) *reinterpret_cast<f32x4*>(dbias + (size_t)s * N + n) = v;
}

// No positions: every sum is zero.
__global__ __launch_bounds__(256) void zero_kernel(float* p, size_t n) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

template <int DT>
static void launch_kind(const ActGradArgs& a, dim3 grid, int per, int shift, hipStream_t s) {
    if (a.act == MOE_ACT_NONE) act_grad_kernel<DT, 0><<<grid, 256, 0, s>>>(a, per, shift);
    else if (a.act == MOE_ACT_SWIGLU) act_grad_kernel<DT, 1><<<grid, 256, 0, s>>>(a, per, shift);
    else act_grad_kernel<DT, 2><<<grid, 256, 0, s>>>(a, per, shift);
}

hipError_t launch_act_grad(const ActGradArgs& a, hipStream_t s) {
    const int S = a.rows.S, R = a.rows.R, N = a.N, I = a.act == MOE_ACT_SWIGLU ? N / 2 : N;
    if (R == 0) {
        if (!a.dbias) return hipSuccess;
        const size_t n = (size_t)S * N;
        zero_kernel<<<dim3((uint32_t)((n + 255) / 256)), 256, 0, s>>>(a.dbias, n);
        return hipGetLastError();
    }
    const int per = part_rows(N, R);
    const int shift = lane_shift(I);
    const long long parts = part_count(S, R, per), chunks = (I + (8 << shift) - 1) / (8 << shift);
    // The columns of a part side by side: what runs at one time reads whole rows (32768 rows of
    // 768, SwiGLU, inputs from HBM: 74.7 us with all parts' first columns first, 71.9 so).
    const dim3 grid((uint32_t)chunks, (uint32_t)parts);
    if (a.dtype == MOE_F32) launch_kind<MOE_F32>(a, grid, per, shift, s);
    else if (a.dtype == MOE_BF16) launch_kind<MOE_BF16>(a, grid, per, shift, s);
    else launch_kind<MOE_F16>(a, grid, per, shift, s);
    // many parts a slot: more lanes (63 parts of 2048 columns 3.4 us by 16 lanes, 5.9 by four; 128
    // slots of three parts on average 6.4 and 4.1)
    int cols = lane_shift(N) + 1;  // lanes of four features, up to 64; fewer, down to 128 bytes, for eight workgroups
    while (cols > 3 && (long long)S * ((N + (4 << cols) - 1) / (4 << cols)) < 8) --cols;
    const dim3 join(S, (N + (4 << cols) - 1) / (4 << cols));
    if (a.dbias && parts > 8ll * S) act_grad_join_kernel<1024><<<join, 1024, 0, s>>>(a.ws, (int)parts, N, cols, a.dbias);
    else if (a.dbias) act_grad_join_kernel<256><<<join, 256, 0, s>>>(a.ws, (int)parts, N, cols, a.dbias);
    return hipGetLastError();
}

}  // namespace qmoe
