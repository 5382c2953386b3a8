// The norm over a list of gradients and their clipping.
//
// Bound by HBM: the norm reads every element once, the clipping reads and writes it.
// 2^29 elements: norm 204 us (bf16, 5.3 TB/s; the conversions to 64 bits show, the largest
// magnitude takes 179) and 354 us (fp32, 6.1 TB/s); clipping bf16 to fp32 532 us (6.1 TB/s),
// fp32 741 us (5.8 TB/s).
// The list travels in the kernel's arguments, up to kNormList or kClipList tensors a
// launch: nothing is copied to the device, and a captured call replays with the same
// addresses.  A longer list whose table the caller keeps on the device takes one launch (317
// tensors of 9000 elements on average, norm and clipping: two launches each 28 us, one each
// 16; a launch takes 4 to 5 us of such tensors however few they are).  A launch's tensors are
// cut into chunks of one size.  Squares
// are summed in 64 bits (at 5 TB/s of fp32 that is 1.3 T fused operations a second of
// the 39 that the card has): neither squares nor sums leave the range.
#include <algorithm>
#include <cmath>

#include "train_ops.h"

namespace qmoe {

constexpr int kNormList = 240, kClipList = 160;  // below 4096 bytes of arguments
constexpr int kGradBlocks = 2048;

// Tensor i's chunks are first[i] .. first[i + 1] (count without one): all of 2^shift elements but
// the last, of tail[i] (bits 0-26); its type stands in bits 28-29, its output's in bits 30-31.
template <int LIST, bool OUT>
struct GradTable {
    const void* in[LIST];
    void* out[OUT ? LIST : 1];
    uint32_t first[LIST];
    uint32_t tail[LIST];
    uint32_t chunks;
    int n, shift;

    __device__ const void* in_at(int i) const { return in[i]; }
    __device__ void* out_at(int i) const { return out[i]; }
    __device__ uint32_t in_type(int i) const { return tail[i] >> 28 & 3; }
    __device__ uint32_t out_type(int i) const { return tail[i] >> 30; }
    __device__ uint32_t first_of(int i) const { return first[i]; }
    __device__ int64_t count_of(int i, uint32_t own) const {
        return ((int64_t)(own - 1) << shift) + (tail[i] & 0x7FFFFFFu);
    }
    // Tensor of chunk c: how many begin at or before it, counted by the wave's lanes in one
    // round of loads (a bisection would be eight, one behind the other).
    __device__ int find(uint32_t c) const {
        const int lane = threadIdx.x & 63;
        int before = 0;
#pragma unroll
        for (int j = 0; j < (LIST + 63) / 64; ++j) {
            const int i = 64 * j + lane;
            before += __popcll(__ballot(i < n && first[min(i, LIST - 1)] <= c));
        }
        return before - 1;
    }
};

// A tensor in a table on the device, empty ones left out.
struct GradEntry {
    void* at;
    int64_t count;      // type in bits 60-61
    uint32_t first[2];  // its first chunk in the norm and in the clipping
};
constexpr int64_t kCountBits = (int64_t(1) << 60) - 1;

template <bool OUT>
struct GradDevice {
    const GradEntry* in;
    const GradEntry* out;
    uint32_t chunks;
    int n, shift;

    __device__ const void* in_at(int i) const { return in[i].at; }
    __device__ void* out_at(int i) const { return out[i].at; }
    __device__ uint32_t in_type(int i) const { return (uint32_t)(in[i].count >> 60); }
    __device__ uint32_t out_type(int i) const { return (uint32_t)(out[i].count >> 60); }
    __device__ uint32_t first_of(int i) const { return in[i].first[OUT]; }
    __device__ int64_t count_of(int i, uint32_t) const { return in[i].count & kCountBits; }
    // As above, in rounds of 64: each lane tests one of 64 places of what is left.
    __device__ int find(uint32_t c) const {
        const int lane = threadIdx.x & 63;
        int from = 0, left = n;
        while (left > 1) {
            const int step = (left + 63) / 64, at = lane * step;
            const int before = __popcll(__ballot(at < left && in[from + min(at, left - 1)].first[OUT] <= c));
            from += (before - 1) * step;
            left = min(step, left - (before - 1) * step);
        }
        return from;
    }
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

// Chunk c of tensor i: its elements (the ones behind the head are cut at multiples of the chunk).
template <typename T>
__device__ __forceinline__ void chunk_range(const T& t, int i, uint32_t c, int head, int64_t& lo, int64_t& hi) {
    const uint32_t first = t.first_of(i), next = i + 1 < t.n ? t.first_of(i + 1) : t.chunks, at = c - first;
    const int64_t n = t.count_of(i, next - first);
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

template <int DT, bool MAX, typename L>
__device__ __forceinline__ void norm_chunk(const L& t, int i, uint32_t c, NormSum& s) {
    typedef typename DType<DT>::type E;
    const E* p = static_cast<const E*>(t.in_at(i));
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

template <bool MAX, typename L>
__global__ __launch_bounds__(256) void grad_norm_kernel(const L t, double* parts) {
    NormSum s = {0.0, 0};
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int i = t.find(c);
        const uint32_t type = t.in_type(i);
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
template <int DI, int DO, typename L>
__device__ __forceinline__ void clip_chunk(const L& t, int i, uint32_t c, float factor) {
    typedef typename DType<DI>::type EI;
    typedef typename DType<DO>::type EO;
    const EI* p = static_cast<const EI*>(t.in_at(i));
    EO* o = static_cast<EO*>(t.out_at(i));
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

template <int DI, typename L>
__device__ __forceinline__ void clip_out(const L& t, int i, uint32_t c, uint32_t out, float f) {
    if (out == MOE_F32) clip_chunk<DI, MOE_F32>(t, i, c, f);
    else if (out == MOE_BF16) clip_chunk<DI, MOE_BF16>(t, i, c, f);
    else clip_chunk<DI, MOE_F16>(t, i, c, f);
}

template <typename L>
__global__ __launch_bounds__(256) void grad_clip_kernel(const L t, const float* total, float max_norm, float eps,
                                                        float scale) {
    // a norm up to max_norm, infinities and 0 included, leaves a factor of 1; NaN stays
    const double norm = (double)total[0] + (double)eps, limit = norm <= (double)max_norm ? 1.0 : (double)max_norm / norm;
    const float factor = (float)((double)scale * limit);
    const uint32_t c = blockIdx.x;
    const int i = t.find(c);
    const uint32_t type = t.in_type(i), out = t.out_type(i);
    if (t.in_at(i) == t.out_at(i) && factor == 1.0f) return;  // in place: nothing changes
    if (type == MOE_F32) clip_out<MOE_F32>(t, i, c, out, factor);
    else if (type == MOE_BF16) clip_out<MOE_BF16>(t, i, c, out, factor);
    else clip_out<MOE_F16>(t, i, c, out, factor);
}

size_t grad_norm_workspace_bytes(int n) {
    return (size_t)std::max(1, (n + kNormList - 1) / kNormList) * kGradBlocks * sizeof(double);
}

// Chunks of 2^12 elements, in the norm up to 2^14 where there are enough for the workgroups
// (204 us of 2^29 elements; 220 in 2^12), more only to keep their number in range.
static int chunk_shift(int64_t total, bool clip) {
    int shift = 12;
    while (shift < (clip ? 12 : 14) && (total >> shift) > 2 * kGradBlocks) ++shift;
    while ((total >> shift) > 1ll << 23) ++shift;  // and with them a launch's threads, below 2^32
    return shift;
}
static uint32_t chunks_of(int64_t count, int shift) { return (uint32_t)((count + (int64_t(1) << shift) - 1) >> shift); }

// The next launch's table: up to LIST tensors that hold elements, from *i on.
template <int LIST, bool OUT>
static void fill_table(const GradListArgs& a, int* i, GradTable<LIST, OUT>& t) {
    int from = *i, to = from, n = 0;
    int64_t total = 0;
    for (; to < a.n && n < LIST; ++to)
        if (a.counts[to] > 0) total += a.counts[to], ++n;
    t.shift = chunk_shift(total, OUT);
    t.n = 0;
    t.chunks = 0;
    for (int j = from; j < to; ++j) {
        const int64_t count = a.counts[j];
        if (count == 0) continue;
        const uint32_t chunks = chunks_of(count, t.shift);
        t.in[t.n] = a.grads[j];
        if (OUT) t.out[t.n] = a.outs ? a.outs[j] : const_cast<void*>(a.grads[j]);
        t.first[t.n] = t.chunks;
        t.tail[t.n] = (uint32_t)(count - ((int64_t)(chunks - 1) << t.shift)) | (uint32_t)a.dtypes[j] << 28 |
                      (uint32_t)(a.outs ? a.out_dtypes[j] : a.dtypes[j]) << 30;
        t.chunks += chunks;
        ++t.n;
    }
    *i = to;
}

size_t grad_table_bytes(int n) { return (size_t)n * sizeof(GradEntry); }

void fill_grad_table(const void* const* at, const int64_t* counts, const int32_t* dtypes, int n, void* table) {
    int64_t total = 0;
    for (int i = 0; i < n; ++i) total += counts[i];
    const int shift[2] = {chunk_shift(total, false), chunk_shift(total, true)};
    uint32_t first[2] = {0, 0};
    GradEntry* e = static_cast<GradEntry*>(table);
    for (int i = 0; i < n; ++i) {
        if (counts[i] == 0) continue;
        *e++ = {const_cast<void*>(at[i]), counts[i] | (int64_t)dtypes[i] << 60, {first[0], first[1]}};
        for (int u = 0; u < 2; ++u) first[u] += chunks_of(counts[i], shift[u]);
    }
}

// The list by its table on the device, if it has one, takes more than one launch without it and is
// not captured (a captured call would need the table at each replay).
template <bool OUT>
static bool use_table(const GradListArgs& a, hipStream_t s, GradDevice<OUT>& t) {
    if (!a.table || a.n <= (OUT ? kClipList : kNormList) || (OUT && a.outs && !a.out_table)) return false;
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s, &capture) != hipSuccess || capture != hipStreamCaptureStatusNone) return false;
    int64_t total = 0;
    for (int i = 0; i < a.n; ++i) total += a.counts[i];
    t = {static_cast<const GradEntry*>(a.table), static_cast<const GradEntry*>(a.outs ? a.out_table : a.table), 0, 0,
         chunk_shift(total, OUT)};
    for (int i = 0; i < a.n; ++i) {
        t.n += a.counts[i] > 0;
        t.chunks += chunks_of(a.counts[i], t.shift);
    }
    return t.n > 0;
}

template <typename L>
static int launch_norm(const GradListArgs& a, const L& t, double* parts, hipStream_t s) {
    const int blocks = (int)std::min<uint32_t>(kGradBlocks, t.chunks);
    if (a.kind == MOE_NORM_MAX) grad_norm_kernel<true><<<blocks, 256, 0, s>>>(t, parts);
    else grad_norm_kernel<false><<<blocks, 256, 0, s>>>(t, parts);
    return blocks;
}

hipError_t launch_grad_norm(const GradListArgs& a, hipStream_t s) {
    double* parts = static_cast<double*>(a.ws);
    int n = 0;
    GradDevice<false> d;
    if (use_table(a, s, d)) {
        n = launch_norm(a, d, parts, s);
    } else {
        for (int i = 0; i < a.n;) {
            GradTable<kNormList, false> t;
            fill_table(a, &i, t);
            if (t.n > 0) n += launch_norm(a, t, parts + n, s);
        }
    }
    const double scale = std::fabs((double)a.scale);
    if (a.kind == MOE_NORM_MAX) grad_total_kernel<true><<<1, 1024, 0, s>>>(parts, n, scale, a.total);
    else grad_total_kernel<false><<<1, 1024, 0, s>>>(parts, n, scale, a.total);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradListArgs& a, hipStream_t s) {
    bool any = false;
    GradDevice<true> d;
    if (use_table(a, s, d)) {
        grad_clip_kernel<<<d.chunks, 256, 0, s>>>(d, a.total, a.max_norm, a.eps, a.scale);
        return hipGetLastError();
    }
    for (int i = 0; i < a.n;) {
        GradTable<kClipList, true> t;
        fill_table(a, &i, t);
        if (t.n == 0) continue;
        grad_clip_kernel<<<t.chunks, 256, 0, s>>>(t, a.total, a.max_norm, a.eps, a.scale);
        any = true;
    }
    return any ? hipGetLastError() : hipSuccess;
}

}  // namespace qmoe
