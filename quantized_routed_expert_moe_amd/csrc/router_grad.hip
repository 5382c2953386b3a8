// The router's balance loss, z loss and per-expert counts over ragged
// sequences, and the gate logits' gradient.
//
// 16 lanes own a row of up to 256 logits, 64 a wider one: it sits in registers, so the
// largest logit, the sums and the probabilities come out of one read, and a sum over a row is
// four steps between lanes for four rows at a time (with 64 lanes for every row the gradient of
// 16384 rows of 256 took 18 us, 10 so: the vector units' time, not the memory's, which is 5 us).
// Losses of those rows: 8.4 us and 4 for the join.
// The probabilities' means are sums over rows in registers, joined over a workgroup's
// waves in LDS, then over workgroups by a second launch in their order: no atomics on
// floats (the counts' are on integers in LDS).
//
// With m the row's largest logit and e = e^(l - m), the probabilities are e / sum e, or
// s / sum s with s = t / (1 + t), t = e e^m: one exponential for both.  The latter is taken as
// r / sum r with r = s for m >= 0 and r = e / (1 + t) = s e^-m for m < 0: rows of low
// logits would underflow in s.
#include <algorithm>

#include "train_ops.h"

namespace qmoe {

constexpr int kLossWaves = 16, kLossThreads = 64 * kLossWaves;

// A row over L lanes: register i of lane l holds element ((i / VEC) * L + l) * VEC + i % VEC.
// VEC = 4 takes 16-byte loads (E a multiple of 4).
template <int L_, int VEC_, int NV_>
struct Row {
    static constexpr int L = L_, VEC = VEC_, NV = NV_, N = VEC * NV, ROWS = 64 / L;  // rows of a wave
    static __device__ __forceinline__ int element(int i, int lane) { return ((i / VEC) * L + lane) * VEC + i % VEC; }
    template <typename T>
    static __device__ __forceinline__ void load(const T* row, int E, int lane, T rest, T* v) {
        typedef T vec __attribute__((ext_vector_type(VEC)));
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            const int e = element(g * VEC, lane);
            vec q;
#pragma unroll
            for (int c = 0; c < VEC; ++c) q[c] = rest;
            if (e < E) q = *reinterpret_cast<const vec*>(row + e);
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[g * VEC + c] = q[c];
        }
    }
};

struct RowSums {
    float m, top;     // largest logit; 0 for -inf (a row of nothing)
    float inv, rinv;  // 1 / sum e, 1 / sum r (0 for a row of nothing)
    float lse;
    float em, rm;     // e^top, and what e / (1 + t) is multiplied by for r
    bool far;         // e^top, or what e loses below its range, matters: the exponential of each logit
};

// e of a logit.  The two roundings of its exponent show as |l - top| 2^-24 of e at most.
__device__ __forceinline__ float exp_from_top(float l, float top) {
    return __builtin_amdgcn_exp2f(1.4426950408889634f * (l - top));
}

// r of a logit given e, and q = 1 - s.
template <bool SIGMOID>
__device__ __forceinline__ float score_of(const RowSums& s, float l, float e, float& q) {
    if (!SIGMOID) {
        q = 1.0f;
        return e;
    }
    if (s.far) {
        const float t = exp_f32(l);
        q = __builtin_amdgcn_rcpf(1.0f + t);
        return s.m < 0.0f ? e * q : t > 1.0f ? 1.0f - q : t * q;
    }
    q = __builtin_amdgcn_rcpf(fmaf(e, s.em, 1.0f));
    return e * s.rm * q;
}

// Of a row's logits l: e, r (SIGMOID; else r is e) and q = 1 - s.  Registers behind the row hold -inf.
template <typename R, bool SIGMOID>
__device__ __forceinline__ RowSums probabilities(const float* l, float* e, float* r, float* q) {
    RowSums s;
    s.m = l[0];
#pragma unroll
    for (int i = 1; i < R::N; ++i) s.m = fmaxf(s.m, l[i]);
    s.m = lanes_max<R::L>(s.m);
    s.top = s.m == -INFINITY ? 0.0f : s.m;
    float sum = 0.0f, rsum = 0.0f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
        e[i] = exp_from_top(l[i], s.top);
        sum += e[i];
    }
    if (SIGMOID) {
        s.far = __any(s.top > 40.0f);
        s.em = exp_f32(s.top);
        s.rm = s.m < 0.0f ? 1.0f : s.em;
        if (s.far) {
#pragma unroll
            for (int i = 0; i < R::N; ++i) rsum += r[i] = score_of<true>(s, l[i], e[i], q[i]);
        } else {
            s.far = false;
#pragma unroll
            for (int i = 0; i < R::N; ++i) {
                q[i] = __builtin_amdgcn_rcpf(fmaf(e[i], s.em, 1.0f));
                rsum += r[i] = e[i] * s.rm * q[i];
            }
        }
        rsum = lanes_sum<R::L>(rsum);
        s.rinv = rsum == 0.0f ? 0.0f : 1.0f / rsum;
    }
    sum = lanes_sum<R::L>(sum);
    s.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    s.lse = sum == 0.0f ? 0.0f : s.top + logf(sum);
    if (!SIGMOID) s.rinv = s.inv;
    return s;
}

struct LossParts {  // the workspace: parts of the rows, [parts][E] sums and counts, [parts] sums of lse^2
    int per, parts;
    float* p;
    int32_t* c;
    float* z;
    float* balance;    // [G * groups of 64 experts]
    int32_t* prefix;   // [G + 1] parts before each sequence
    int32_t* done;     // workgroups of the second launch that have ended
};

// Rows of all sequences and of sequence g.
__device__ __forceinline__ int rows_of_all(const RowMap& m) {
    if (!m.offsets) return m.R;
    const int a = min(max(m.offsets[0], 0), m.R), b = min(max(m.offsets[m.S], 0), m.R);
    return max(b - a, 0);
}

// Sum over the workgroup, in a fixed order, in every thread.
template <int WAVES>
__device__ __forceinline__ float group_sum(float v) {
    __shared__ float part[WAVES];
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += part[w];
    return s;
}

// One part of the rows: sums of the probabilities, counts and sum of lse^2.
// ALONE: there is one part only, and the workgroup writes the results.
template <typename R, bool SIGMOID, bool ALONE>
__global__ __launch_bounds__(kLossThreads) void loss_rows_kernel(const RouterArgs a, const LossParts ws) {
    constexpr int WIDE = R::N * R::L;  // elements that the registers hold
    __shared__ float join[kLossWaves * WIDE];
    __shared__ int hist[1024];
    const int lane = threadIdx.x % R::L, unit = threadIdx.x / R::L, wave = threadIdx.x >> 6, E = a.E;
    hist[threadIdx.x] = 0;
    int seq, q0, nq;
    if (ALONE) {
        const int2 r = slot_range(a.seqs, 0);
        q0 = r.x;
        nq = r.y;
    } else {
        if (blockIdx.x == 0 && threadIdx.x == 0) *ws.done = 0;
        if (!find_part<kLossThreads>(a.seqs, ws.per, blockIdx.x, blockIdx.x == 0 ? ws.prefix : nullptr, seq, q0, nq)) return;
    }
    // the first ids, requested ahead of the rows
    const int32_t* ids = a.ids + (size_t)q0 * a.k;
    const int early = (int)threadIdx.x < nq * a.k ? ids[threadIdx.x] : -1;
    float acc[R::N] = {}, z = 0.0f;
    for (int r0 = 0; r0 < nq; r0 += kLossWaves * R::ROWS) {
        const int row = r0 + unit;
        const bool live = row < nq;
        float l[R::N], e[R::N], r[R::N], q[R::N];
        R::load(a.logits + (size_t)(q0 + min(row, nq - 1)) * E, E, lane, -INFINITY, l);
        const RowSums s = probabilities<R, SIGMOID>(l, e, r, q);
        const float inv = live ? s.rinv : 0.0f;  // the row behind the last is the last once more
#pragma unroll
        for (int i = 0; i < R::N; ++i) acc[i] = fmaf(SIGMOID ? r[i] : e[i], inv, acc[i]);
        z = live ? fmaf(s.lse, s.lse, z) : z;
    }
    __syncthreads();  // hist is cleared
    if (early >= 0 && early < E) atomicAdd(&hist[early], 1);
    for (int i = threadIdx.x + kLossThreads; i < nq * a.k; i += kLossThreads) {
        const int id = ids[i];
        if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
    }
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
        const float v = R::L == 16 ? sum_of_rows(acc[i]) : acc[i];
        if (R::L == 64 || (threadIdx.x & 63) < 16) join[wave * WIDE + R::element(i, lane)] = v;
    }
    z = group_sum<kLossWaves>(lane == 0 ? z : 0.0f);
    __syncthreads();
    const int e = threadIdx.x;
    float sum = 0.0f;
    if (e < E)
        for (int w = 0; w < kLossWaves; ++w) sum += join[w * WIDE + e];
    if (ALONE) {
        const float mean = nq > 0 ? sum / (float)nq : 0.0f;
        const float balance = group_sum<kLossWaves>(e < E ? (float)hist[e] * mean : 0.0f);
        if (e < E) {
            a.counts_out[e] = hist[e];
            a.probs[e] = mean;
        }
        if (e == 0) {
            a.losses[0] = nq > 0 ? balance * ((float)E / ((float)a.k * (float)nq)) : 0.0f;
            a.losses[1] = nq > 0 ? z / (float)nq : 0.0f;
        }
    } else {
        if (e < E) {
            ws.p[(size_t)blockIdx.x * E + e] = sum;
            ws.c[(size_t)blockIdx.x * E + e] = hist[e];
        }
        if (e == 0) ws.z[blockIdx.x] = z;
    }
}

// Counts and means of 64 experts of a sequence: 64 columns by 16 lanes of parts.  The
// workgroup that ends last adds the losses' parts, in their order.
__global__ __launch_bounds__(1024) void loss_join_kernel(const RouterArgs a, const LossParts ws) {
    __shared__ float sp[1024];
    __shared__ int sc[1024], last;
    const int g = blockIdx.x, e = blockIdx.y * 64 + (threadIdx.x & 63), lane = threadIdx.x >> 6, E = a.E;
    const int from = ws.prefix[g], to = min(ws.prefix[g + 1], ws.parts), n = slot_range(a.seqs, g).y;
    float p = 0.0f;
    int c = 0;
    if (e < E)
        for (int i = from + lane; i < to; i += 16) {
            p += ws.p[(size_t)i * E + e];
            c += ws.c[(size_t)i * E + e];
        }
    sp[threadIdx.x] = p;
    sc[threadIdx.x] = c;
    __syncthreads();
    const int groups = gridDim.y, total = gridDim.x * groups;
    if (lane == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            p += sp[threadIdx.x + 64 * i];
            c += sc[threadIdx.x + 64 * i];
        }
        const float mean = n > 0 ? p / (float)n : 0.0f;
        if (e < E) {
            a.counts_out[(size_t)g * E + e] = c;
            a.probs[(size_t)g * E + e] = mean;
        }
        const float b = wave_sum(e < E ? (float)c * mean : 0.0f);
        if (threadIdx.x == 0) {
            __hip_atomic_store(ws.balance + g * groups + blockIdx.y, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(ws.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    float b = 0.0f, z = 0.0f;
    for (int i = threadIdx.x; i < total; i += 1024)
        b += __hip_atomic_load(ws.balance + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int parts = min(ws.prefix[a.seqs.S], ws.parts), rows = rows_of_all(a.seqs);
    for (int i = threadIdx.x; i < parts; i += 1024) z += ws.z[i];
    b = group_sum<16>(b);
    z = group_sum<16>(z);
    if (threadIdx.x == 0) {
        a.losses[0] = rows > 0 ? b * ((float)E / ((float)a.k * (float)rows)) : 0.0f;
        a.losses[1] = rows > 0 ? z / (float)rows : 0.0f;
    }
}

// Rows of a part: what a workgroup's waves hold at a time until there are 512 parts, of wide rows
// 256 (4096 rows of 1024: 19.6 us in parts of 64, 14.4 in 16; 16384 of 1000: 24 in 64, 30 in 32).
static int least_rows(int E) { return E <= 256 ? 64 : 16; }
static int most_parts(int E) { return E <= 256 ? 512 : 256; }
static int loss_rows(int T, int E) {
    int per = least_rows(E);
    while (T / per > most_parts(E)) per *= 2;
    return per;
}

// whole: parts of `per` rows in all; beside them each sequence may begin one.
static LossParts loss_parts(int whole, int T, int E, int G, void* ws, size_t* bytes) {
    LossParts l{};
    l.parts = whole + (G < T ? G : T) + (T == 0);  // one at least: it writes the prefix
    const size_t groups = (E + 63) / 64;
    size_t at = 0;
    auto take = [&](size_t n) {
        void* p = ws ? static_cast<uint8_t*>(ws) + at : nullptr;
        at += (n * 4 + 15) / 16 * 16;
        return p;
    };
    l.p = static_cast<float*>(take((size_t)l.parts * E));
    l.c = static_cast<int32_t*>(take((size_t)l.parts * E));
    l.z = static_cast<float*>(take(l.parts));
    l.balance = static_cast<float*>(take(G * groups));
    l.prefix = static_cast<int32_t*>(take(G + 1));
    l.done = static_cast<int32_t*>(take(1));
    if (bytes) *bytes = at;
    return l;
}

// The parts' number falls where their rows double, and from 256 experts to 257; the need does
// not: it is that of the most parts of any T up to this one, and for wide rows that of 256 experts at least.
size_t balance_loss_workspace_bytes(int T, int E, int G) {
    size_t bytes = 0, narrow = 0;
    loss_parts(std::min(T / least_rows(E), most_parts(E)), T, E, G, nullptr, &bytes);
    if (E > 256) loss_parts(std::min(T / least_rows(256), most_parts(256)), T, 256, G, nullptr, &narrow);
    return std::max(bytes, narrow);
}

template <typename R>
static void launch_loss_rows(const RouterArgs& a, const LossParts& ws, bool alone, hipStream_t s) {
    const dim3 grid(alone ? 1 : ws.parts);
    if (a.score == MOE_SCORE_SIGMOID) {
        if (alone) loss_rows_kernel<R, true, true><<<grid, kLossThreads, 0, s>>>(a, ws);
        else loss_rows_kernel<R, true, false><<<grid, kLossThreads, 0, s>>>(a, ws);
    } else {
        if (alone) loss_rows_kernel<R, false, true><<<grid, kLossThreads, 0, s>>>(a, ws);
        else loss_rows_kernel<R, false, false><<<grid, kLossThreads, 0, s>>>(a, ws);
    }
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// launch(Row) with the smallest row that holds E logits.
template <typename F>
static void by_width(int E, bool wide, F&& launch) {
    if (wide) {
        if (E <= 64) launch(Row<16, 4, 1>{});
        else if (E <= 128) launch(Row<16, 4, 2>{});
        else if (E <= 256) launch(Row<16, 4, 4>{});
        else if (E <= 512) launch(Row<64, 4, 2>{});
        else launch(Row<64, 4, 4>{});
    } else {
        if (E <= 64) launch(Row<16, 1, 4>{});
        else if (E <= 256) launch(Row<16, 1, 16>{});
        else launch(Row<64, 1, 16>{});
    }
}

hipError_t launch_balance_loss(const RouterArgs& a, hipStream_t s) {
    const int G = a.seqs.S, groups = (a.E + 63) / 64;
    const int per = loss_rows(a.T, a.E);
    LossParts ws = loss_parts(a.T / per, a.T, a.E, G, a.ws, nullptr);
    ws.per = per;
    const bool alone = G == 1 && a.T <= 64;
    by_width(a.E, a.E % 4 == 0 && aligned16(a.logits), [&](auto row) { launch_loss_rows<decltype(row)>(a, ws, alone, s); });
    if (!alone) loss_join_kernel<<<dim3(G, groups), 1024, 0, s>>>(a, ws);
    return hipGetLastError();
}

// --------------------------------------------------------------- gradient

// Sequences of the rows t0 .. t0 + ROWS of a wave, that of this lane's row: the last one that
// begins at or before it, -1 if it lies in none.
template <typename R>
__device__ __forceinline__ int sequence_of(const RowMap& m, int t0) {
    if (!m.offsets) return 0;
    // 64 places first, then the ones behind the last that fits (262144 rows of 64 in 1024 sequences:
    // 81 us by a count of all offsets, 52 so).
    const int lane = threadIdx.x & 63, step = m.S / 64 + 1;
    const int at = m.offsets[min(lane * step, m.S)];
    int before[R::ROWS];
#pragma unroll
    for (int r = 0; r < R::ROWS; ++r) before[r] = __popcll(__ballot(lane * step <= m.S && at <= t0 + r));
    if (step > 1) {
#pragma unroll
        for (int r = 0; r < R::ROWS; ++r) {
            const int base = max(before[r] - 1, 0) * step, i = base + lane;
            const bool in = lane < step && i <= m.S && m.offsets[min(i, m.S)] <= t0 + r;
            before[r] = base + __popcll(__ballot(in));
        }
    }
    int mine = before[0];
#pragma unroll
    for (int r = 1; r < R::ROWS; ++r) mine = lane / R::L == r ? before[r] : mine;
    return mine >= 1 && mine <= m.S ? mine - 1 : -1;
}

// f(integral constants 0 .. N - 1).
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unrolled<N, I + 1>(f);
    }
}

// The lanes write the row's gradient through the losses (and, of a softmax that is not
// renormalised, the pull of the weights' sum); then lane j of them, which holds pair j (and j + L,
// ...), writes its expert's logit once more, with all that comes from the pairs of this
// expert, and the rest computed again from the logit.  (Adding the pairs' terms to the registers
// that hold their logits took a third of the kernel.)  A wave's stores to one place are made in
// their order.
template <typename R, int KP, bool SIGMOID, int OUT>
__global__ __launch_bounds__(256) void route_grad_kernel(const RouterArgs a) {
    constexpr int N = R::N, L = R::L;
    const int lane = threadIdx.x % L, E = a.E, k = a.k;
    const int t0 = (blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * R::ROWS;
    if (t0 >= a.T) return;
    const bool live = t0 + (int)(threadIdx.x & 63) / L < a.T;
    const int t = min(t0 + (int)(threadIdx.x & 63) / L, a.T - 1);
    const float* row = a.logits + (size_t)t * E;
    const bool pull = a.dw && !SIGMOID && !a.renormalize;  // the weights depend on all logits
    const bool whole = a.counts || pull;

    // the pairs
    int id[KP];
    float dw[KP], z[KP];
    bool valid[KP];
#pragma unroll
    for (int u = 0; u < KP; ++u) {
        const int j = u * L + lane;
        id[u] = a.dw && j < k ? a.ids[(size_t)t * k + j] : -1;
        valid[u] = id[u] >= 0 && id[u] < E;
        dw[u] = valid[u] ? a.scale * a.dw[(size_t)t * k + j] : 0.0f;
        z[u] = valid[u] ? row[id[u]] : -INFINITY;
    }
    float l[N], e[N], r[N], q[N], f[N];
    RowSums s = {};
    int seq = -1;
    float b = 0.0f, zs = 0.0f, dot = 0.0f, draw = 0.0f;
    const int32_t* counts = a.counts;
    if (whole) R::load(row, E, lane, -INFINITY, l);
    if (a.counts) {
        seq = sequence_of<R>(a.seqs, t0);
        counts += (size_t)max(seq, 0) * E;
        int32_t c[N];
        R::load(counts, E, lane, 0, c);
        const float n = (float)rows_of_all(a.seqs), ng = (float)slot_range(a.seqs, max(seq, 0)).y;
        b = a.dlosses[0] * ((float)E / ((float)k * n)) / ng;
        zs = a.dlosses[1] * (2.0f / n);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = (float)c[i];
    }
    if (whole) s = probabilities<R, SIGMOID>(l, e, r, q);
    if (a.counts) {
#pragma unroll
        for (int i = 0; i < N; ++i) dot = fmaf(SIGMOID ? r[i] : e[i], f[i], dot);
        dot = lanes_sum<L>(dot) * s.rinv;
        b *= s.rinv;
        zs *= s.lse * s.inv;
    }

    // the weights' part: each pair's own term, and the pull on every logit
    float term[KP];
    if (a.dw) {
        float u[KP], sum = 0.0f, mean = 0.0f, m = -INFINITY;
#pragma unroll
        for (int i = 0; i < KP; ++i) m = fmaxf(m, z[i]);
        if (a.renormalize) m = lanes_max<L>(m);
        const float top = a.renormalize ? (m == -INFINITY ? 0.0f : m) : s.top;
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            if (SIGMOID) u[i] = a.renormalize && m < 0.0f ? exp_down(z[i] - top) * sigmoid_f32(-z[i]) : sigmoid_f32(z[i]);
            else u[i] = exp_down(z[i] - top);
            sum += u[i];
        }
        if (a.renormalize) sum = lanes_sum<L>(sum);
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            // divided: the weight of a single expert is 1 exactly, its gradient 0
            if (a.renormalize) u[i] = sum == 0.0f ? 0.0f : u[i] / sum;
            else if (!SIGMOID) u[i] *= s.inv;
            if (!valid[i]) u[i] = 0.0f;
            mean += valid[i] ? u[i] * dw[i] : 0.0f;
        }
        mean = a.renormalize || !SIGMOID ? lanes_sum<L>(mean) : 0.0f;
        if (!a.renormalize) {
            draw = mean * s.inv;  // of every logit (0 for SIGMOID)
            mean = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            term[i] = valid[i] ? u[i] * (dw[i] - mean) : 0.0f;
            if (SIGMOID) term[i] = valid[i] ? term[i] * sigmoid_f32(-z[i]) : 0.0f;
        }
    }

    typedef typename DType<OUT>::type T;
    T* out = static_cast<T*>(a.dlogits) + (size_t)t * E;
    // the part that all logits have
    auto common = [&](float e, float r, float q, float f) {
        float d = pull ? -e * draw : 0.0f;
        if (seq >= 0) d += fmaf(r * b, (f - dot) * q, zs * e);
        return d;
    };
#pragma unroll
    for (int g = 0; g < R::NV; ++g) {
        const int at = R::element(g * R::VEC, lane);
        typedef T vec __attribute__((ext_vector_type(R::VEC)));
        vec v;
#pragma unroll
        for (int c = 0; c < R::VEC; ++c) {
            const int i = g * R::VEC + c;
            v[c] = (T)(whole ? common(e[i], SIGMOID ? r[i] : e[i], SIGMOID ? q[i] : 1.0f, f[i]) : 0.0f);
        }
        if (live && at < E) *reinterpret_cast<vec*>(out + at) = v;
    }
    if (!a.dw) return;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    float all[KP] = {};
#pragma unroll
    for (int w = 0; w < KP; ++w)
        unrolled<L>([&](auto tag) {
            constexpr int J = decltype(tag)::value;
            if (w * L + J >= k) return;
            const int other = lanes_get<L, J>(id[w]);
            const float v = __int_as_float(lanes_get<L, J>(__float_as_int(term[w])));
#pragma unroll
            for (int u = 0; u < KP; ++u) all[u] += other == id[u] ? v : 0.0f;
        });
#pragma unroll
    for (int u = 0; u < KP; ++u) {
        float d = all[u];
        if (whole) {
            const float ez = exp_from_top(z[u], s.top), count = a.counts && valid[u] ? (float)counts[id[u]] : 0.0f;
            float qz;
            const float rz = score_of<SIGMOID>(s, z[u], ez, qz);
            d += common(ez, rz, qz, count);
        }
        if (live && valid[u]) out[id[u]] = (T)d;
    }
}

template <typename R, int KP>
static void launch_route_grad(const RouterArgs& a, hipStream_t s) {
    const dim3 grid((a.T + 4 * R::ROWS - 1) / (4 * R::ROWS));
    auto go = [&](auto sig, auto out) {
        route_grad_kernel<R, KP, decltype(sig)::value, decltype(out)::value><<<grid, 256, 0, s>>>(a);
    };
    auto type = [&](auto sig) {
        if (a.out_dtype == MOE_F32) go(sig, std::integral_constant<int, MOE_F32>{});
        else if (a.out_dtype == MOE_BF16) go(sig, std::integral_constant<int, MOE_BF16>{});
        else go(sig, std::integral_constant<int, MOE_F16>{});
    };
    if (a.score == MOE_SCORE_SIGMOID) type(std::true_type{});
    else type(std::false_type{});
}

hipError_t launch_route_backward(const RouterArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const bool wide = a.E % 4 == 0 && aligned16(a.logits) && aligned16(a.dlogits) && aligned16(a.counts);
    by_width(a.E, wide, [&](auto row) {
        typedef decltype(row) R;
        if constexpr (R::L == 16) {
            if (a.k > 16) return launch_route_grad<R, 4>(a, s);
        }
        launch_route_grad<R, 1>(a, s);
    });
    return hipGetLastError();
}

}  // namespace qmoe
