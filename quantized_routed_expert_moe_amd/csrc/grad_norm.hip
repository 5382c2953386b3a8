// The norm over a list of gradients and their clipping.
//
// Bound by HBM: the norm reads every element once, the clipping reads and writes it.
// 2^29 elements: norm 204 us (bf16, 5.3 TB/s; the conversions to 64 bits show, the largest
// magnitude takes 179) and 354 us (fp32, 6.1 TB/s); clipping bf16 to fp32 532 us (6.1 TB/s),
// fp32 741 us (5.8 TB/s).
// The list travels in the kernel's arguments, up to kNormList or kClipList tensors a
// launch: nothing is copied to the device, and a captured call replays with the same
// addresses.  A launch's tensors are cut into chunks of one size.  Squares
// are summed in 64 bits (at 5 TB/s of fp32 that is 1.3 T fused operations a second of
// the 39 that the card has): neither squares nor sums leave the range.
#include <algorithm>
#include <cmath>

#include "train_ops.h"

namespace qmoe {

constexpr int kNormList = 240, kClipList = 160;  // below 4096 bytes of arguments
constexpr int kGradBlocks = 2048;

// Tensor i's chunks are first[i] .. first[i + 1] (count without one): all of `chunk` elements
// but the last, of tail[i] (bits 0-26); its type stands in bits 28-29, its output's in bits 30-31.
template <int LIST, bool OUT>
struct GradTable {
    const void* in[LIST];
    void* out[OUT ? LIST : 1];
    uint32_t first[LIST];
    uint32_t tail[LIST];
    uint32_t chunks;
    int n, shift;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__bf16 v) { return (float)v; }
__device__ __forceinline__ float to_float(_Float16 v) { return (float)v; }

constexpr int kUnroll = 4;  // vectors that a thread has in flight

// Elements [lo, hi) of a chunk, given the number of elements of the tensor's head (before
// the first 16-byte boundary): vectors of W by `vec`, kUnroll of them a turn 256 W apart (at and
// below end), the rest by `one`.
template <int W, typename V, typename O>
__device__ __forceinline__ void walk(int64_t lo, int64_t hi, int head, bool vectors, V&& vec, O&& one) {
    if (!vectors) {
        for (int64_t i = lo + threadIdx.x; i < hi; i += 256) one(i);
        return;
    }
    const int64_t start = lo < head ? min((int64_t)head, hi) : lo;
    for (int64_t i = lo + threadIdx.x; i < start; i += 256) one(i);
    const int64_t end = start + (hi - start) / W * W;
    for (int64_t i = start + threadIdx.x * W; i < end; i += kUnroll * 256 * W) vec(i, end);
    for (int64_t i = end + threadIdx.x; i < hi; i += 256) one(i);
}

// Tensor of chunk c: how many begin at or before it, counted by the wave's lanes in one round
// of loads (a bisection would be eight, one behind the other).
template <int LIST, bool OUT>
__device__ __forceinline__ int tensor_of(const GradTable<LIST, OUT>& t, uint32_t c) {
    const int lane = threadIdx.x & 63;
    int before = 0;
#pragma unroll
    for (int j = 0; j < (LIST + 63) / 64; ++j) {
        const int i = 64 * j + lane;
        before += __popcll(__ballot(i < t.n && t.first[min(i, LIST - 1)] <= c));
    }
    return before - 1;
}

// Chunk c of tensor i: its elements (the ones behind the head are cut at multiples of the chunk).
template <typename T>
__device__ __forceinline__ void chunk_range(const T& t, int i, uint32_t c, int head, int64_t& lo, int64_t& hi) {
    const uint32_t first = t.first[i], next = i + 1 < t.n ? t.first[i + 1] : t.chunks, at = c - first;
    const int64_t n = ((int64_t)(next - first - 1) << t.shift) + (t.tail[i] & 0x7FFFFFFu);
    lo = at == 0 ? 0 : min(n, ((int64_t)at << t.shift) + head);
    hi = c + 1 == next ? n : min(n, ((int64_t)(at + 1) << t.shift) + head);
}

// Elements before the first 16-byte boundary.
template <typename E>
__device__ __forceinline__ int head_of(const void* p) {
    return (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(E);
}

struct NormSum {
    double sum;      // of squares
    uint32_t most;   // magnitude bits: NaN above infinity above all else
};

template <int DT, bool MAX>
__device__ __forceinline__ void norm_chunk(const GradTable<kNormList, false>& t, int i, uint32_t c, NormSum& s) {
    typedef typename DType<DT>::type E;
    const E* p = static_cast<const E*>(t.in[i]);
    const int head = head_of<E>(p);
    int64_t lo, hi;
    chunk_range(t, i, c, head, lo, hi);
    auto add = [&](float v) {
        if (MAX) s.most = max(s.most, __float_as_uint(v) & 0x7FFFFFFFu);
        else s.sum = fma((double)v, (double)v, s.sum);
    };
    walk<8>(lo, hi, head, true,
         [&](int64_t at, int64_t end) {
             float v[kUnroll][8] = {};
#pragma unroll
             for (int u = 0; u < kUnroll; ++u)
                 if (at + u * 2048 < end) load_vec8<DT>(p, at + u * 2048, v[u]);
#pragma unroll
             for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                 for (int j = 0; j < 8; ++j) add(v[u][j]);
         },
         [&](int64_t at) { add(to_float(p[at])); });
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ uint32_t wave_most(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}

// Sum (or largest) over the workgroup, in thread 0.
template <int WAVES, bool MAX>
__device__ __forceinline__ double group_norm(NormSum s) {
    __shared__ double part[WAVES];
    const double v = MAX ? (double)wave_most(s.most) : wave_sum64(s.sum);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) r = MAX ? max(r, part[w]) : r + part[w];
    return r;
}

template <bool MAX>
__global__ __launch_bounds__(256) void grad_norm_kernel(const GradTable<kNormList, false> t, double* parts) {
    NormSum s = {0.0, 0};
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const uint32_t type = t.tail[i] >> 28 & 3;
        if (type == MOE_F32) norm_chunk<MOE_F32, MAX>(t, i, c, s);
        else if (type == MOE_BF16) norm_chunk<MOE_BF16, MAX>(t, i, c, s);
        else norm_chunk<MOE_F16, MAX>(t, i, c, s);
    }
    const double v = group_norm<4, MAX>(s);
    if (threadIdx.x == 0) parts[blockIdx.x] = v;
}

// total of the parts of all launches.
template <bool MAX>
__global__ __launch_bounds__(1024) void grad_total_kernel(const double* parts, int n, double scale, float* total) {
    NormSum s = {0.0, 0};
    for (int i = threadIdx.x; i < n; i += 1024) {
        if (MAX) s.most = max(s.most, (uint32_t)parts[i]);
        else s.sum += parts[i];
    }
    const double v = group_norm<16, MAX>(s);
    if (threadIdx.x == 0) total[0] = (float)(scale * (MAX ? (double)__uint_as_float((uint32_t)v) : sqrt(v)));
}

// A chunk is one or two turns of a workgroup, and there is a workgroup for each: all of them
// then sweep the memory together (bf16 to fp32, 2^29 elements: 605 us by 2048 workgroups that
// take such chunks in turn, 623 with chunks of 2^16, 532 so).  Loads and stores go past the
// caches: 532 us, 563 through them (2^24 elements, norm and clipping 26 and 32 us).  A vector
// is 16 bytes of the wider type, so that a wave's accesses are whole runs (682 and 620 us).
template <int DI, int DO>
__device__ __forceinline__ void clip_chunk(const GradTable<kClipList, true>& t, int i, uint32_t c, float factor) {
    typedef typename DType<DI>::type EI;
    typedef typename DType<DO>::type EO;
    const EI* p = static_cast<const EI*>(t.in[i]);
    EO* o = static_cast<EO*>(t.out[i]);
    const int head = head_of<EI>(p);
    int64_t lo, hi;
    chunk_range(t, i, c, head, lo, hi);
    const bool vectors = head_of<EO>(o + head) == 0;
    constexpr int W = DI == MOE_F32 || DO == MOE_F32 ? 4 : 8;
    typedef EI in_t __attribute__((ext_vector_type(W)));
    typedef EO out_t __attribute__((ext_vector_type(W)));
    walk<W>(lo, hi, head, vectors,
            [&](int64_t at, int64_t end) {
                in_t v[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
                    if (at + u * 256 * W < end)
                        v[u] = __builtin_nontemporal_load(reinterpret_cast<const in_t*>(p + at + u * 256 * W));
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (at + u * 256 * W >= end) continue;
                    out_t r;
#pragma unroll
                    for (int j = 0; j < W; ++j) r[j] = (EO)((float)v[u][j] * factor);
                    out_t* to = reinterpret_cast<out_t*>(o + at + u * 256 * W);
                    __builtin_nontemporal_store(r, to);
                }
            },
            [&](int64_t at) { o[at] = (EO)(to_float(p[at]) * factor); });
}

template <int DI>
__device__ __forceinline__ void clip_out(const GradTable<kClipList, true>& t, int i, uint32_t c, uint32_t out, float f) {
    if (out == MOE_F32) clip_chunk<DI, MOE_F32>(t, i, c, f);
    else if (out == MOE_BF16) clip_chunk<DI, MOE_BF16>(t, i, c, f);
    else clip_chunk<DI, MOE_F16>(t, i, c, f);
}

__global__ __launch_bounds__(256) void grad_clip_kernel(const GradTable<kClipList, true> t, const float* total,
                                                        float max_norm, float eps, float scale) {
    const double norm = (double)total[0] + (double)eps, limit = norm == 0.0 ? 1.0 : (double)max_norm / norm;
    const float factor = (float)((double)scale * (limit > 1.0 ? 1.0 : limit));  // NaN stays
    const uint32_t c = blockIdx.x;
    const int i = tensor_of(t, c);
    const uint32_t type = t.tail[i] >> 28 & 3, out = t.tail[i] >> 30;
    if (t.in[i] == t.out[i] && factor == 1.0f) return;  // in place: nothing changes
    if (type == MOE_F32) clip_out<MOE_F32>(t, i, c, out, factor);
    else if (type == MOE_BF16) clip_out<MOE_BF16>(t, i, c, out, factor);
    else clip_out<MOE_F16>(t, i, c, out, factor);
}

size_t grad_norm_workspace_bytes(int n) {
    return (size_t)std::max(1, (n + kNormList - 1) / kNormList) * kGradBlocks * sizeof(double);
}

// The next launch's table: up to LIST tensors that hold elements, from *i on.  Chunks of 2^12
// elements, up to 2^most where there are enough for the workgroups (the norm takes 204 us in
// chunks of 2^14, 220 in 2^12), more only to keep their number in range.
template <int LIST, bool OUT>
static void fill_table(const GradListArgs& a, int* i, int most, GradTable<LIST, OUT>& t) {
    int from = *i, to = from, n = 0;
    int64_t total = 0;
    for (; to < a.n && n < LIST; ++to)
        if (a.counts[to] > 0) total += a.counts[to], ++n;
    t.shift = 12;
    while (t.shift < most && (total >> t.shift) > 2 * kGradBlocks) ++t.shift;
    while ((total >> t.shift) > 1ll << 30) ++t.shift;
    t.n = 0;
    t.chunks = 0;
    for (int j = from; j < to; ++j) {
        const int64_t count = a.counts[j];
        if (count == 0) continue;
        const int64_t chunks = (count + (int64_t(1) << t.shift) - 1) >> t.shift;
        t.in[t.n] = a.grads[j];
        if (OUT) t.out[t.n] = a.outs ? a.outs[j] : const_cast<void*>(a.grads[j]);
        t.first[t.n] = t.chunks;
        t.tail[t.n] = (uint32_t)(count - ((chunks - 1) << t.shift)) | (uint32_t)a.dtypes[j] << 28 |
                      (uint32_t)(a.outs ? a.out_dtypes[j] : a.dtypes[j]) << 30;
        t.chunks += (uint32_t)chunks;
        ++t.n;
    }
    *i = to;
}

hipError_t launch_grad_norm(const GradListArgs& a, hipStream_t s) {
    double* parts = static_cast<double*>(a.ws);
    int n = 0;
    for (int i = 0; i < a.n;) {
        GradTable<kNormList, false> t;
        fill_table(a, &i, 14, t);
        if (t.n == 0) continue;
        const int blocks = (int)std::min<uint32_t>(kGradBlocks, t.chunks);
        if (a.kind == MOE_NORM_MAX) grad_norm_kernel<true><<<blocks, 256, 0, s>>>(t, parts + n);
        else grad_norm_kernel<false><<<blocks, 256, 0, s>>>(t, parts + n);
        n += blocks;
    }
    const double scale = std::fabs((double)a.scale);
    if (a.kind == MOE_NORM_MAX) grad_total_kernel<true><<<1, 1024, 0, s>>>(parts, n, scale, a.total);
    else grad_total_kernel<false><<<1, 1024, 0, s>>>(parts, n, scale, a.total);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradListArgs& a, hipStream_t s) {
    bool any = false;
    for (int i = 0; i < a.n;) {
        GradTable<kClipList, true> t;
        fill_table(a, &i, 12, t);
        if (t.n == 0) continue;
        grad_clip_kernel<<<t.chunks, 256, 0, s>>>(t, a.total, a.max_norm, a.eps, a.scale);
        any = true;
    }
    return any ? hipGetLastError() : hipSuccess;
}

}  // namespace qmoe
