// The router's balance loss, z loss and per-expert counts over ragged
// sequences, and the gate logits' gradient.
//
// A wave owns a row: its E <= 1024 logits sit in registers, so the largest logit,
// the sums and the probabilities come out of one read.  Rows are a few KB, so
// short calls are latency and long ones HBM (logits once, and the gradient once).
// The probabilities' means are sums over rows in registers, joined over a workgroup's
// waves in LDS, then over workgroups by a second launch in their order: no atomics on
// floats (the counts' are on integers in LDS).
//
// With m the row's largest logit, s = sigmoid(l) and e = e^(l - m), the
// probabilities are e / sum e, or s / sum s.  The latter is taken as r / sum r with
// r = s for m >= 0 and r = e sigmoid(-l) = s e^-m for m < 0: rows of low logits
// would underflow in s.
#include "train_ops.h"

namespace qmoe {

constexpr int kLossWaves = 16, kLossThreads = 64 * kLossWaves;

// A row in registers: register i of lane l holds element ((i / VEC) * 64 + l) * VEC + i % VEC.
// VEC = 4 takes 16-byte loads (E a multiple of 4).
template <int VEC, int NV>
struct Row {
    static constexpr int N = VEC * NV;
    static __device__ __forceinline__ int element(int i, int lane) { return ((i / VEC) * 64 + lane) * VEC + i % VEC; }
    static __device__ __forceinline__ void load(const float* row, int E, int lane, float* v) {
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            const int e = element(g * VEC, lane);
            if constexpr (VEC == 4) {
                const float4 q = e < E ? *reinterpret_cast<const float4*>(row + e)
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                v[4 * g] = q.x; v[4 * g + 1] = q.y; v[4 * g + 2] = q.z; v[4 * g + 3] = q.w;
            } else {
                v[g] = e < E ? row[e] : -INFINITY;
            }
        }
    }
};

// Probabilities of a row.  p: as above; soft: softmax (of SIGMOID rows too), e^(l - top) inv;
// lse: log of the sum of e^l.  Registers behind the row hold -inf and come out as 0.
template <int N, bool SIGMOID>
__device__ __forceinline__ void probabilities(const float* l, float* p, float* soft, float& lse, float& top, float& inv) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
    top = m == -INFINITY ? 0.0f : m;  // a row of nothing
    float sum = 0.0f, rsum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        soft[i] = exp_f32(l[i] - top);
        sum += soft[i];
        if (SIGMOID) {
            p[i] = m < 0.0f ? soft[i] * sigmoid_f32(-l[i]) : sigmoid_f32(l[i]);
            rsum += p[i];
        }
    }
    sum = wave_sum(sum);
    lse = sum == 0.0f ? 0.0f : top + logf(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (SIGMOID) rsum = wave_sum(rsum);
    const float rinv = rsum == 0.0f ? 0.0f : 1.0f / rsum;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        soft[i] *= inv;
        p[i] = SIGMOID ? p[i] * rinv : soft[i];
    }
}

struct LossParts {  // the workspace: parts of the rows, [parts][E] sums and counts, [parts] sums of lse^2
    int per, parts;
    float* p;
    int32_t* c;
    float* z;
    float* balance;    // [G * groups of 64 experts]
    int32_t* prefix;   // [G + 1] parts before each sequence
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
template <int VEC, int NV, bool SIGMOID, bool ALONE>
__global__ __launch_bounds__(kLossThreads) void loss_rows_kernel(const RouterArgs a, const LossParts ws) {
    typedef Row<VEC, NV> R;
    __shared__ float join[kLossWaves * R::N * 64];
    __shared__ int hist[1024];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E;
    hist[threadIdx.x] = 0;
    int seq, q0, nq;
    const bool any = find_part<kLossThreads>(a.seqs, ws.per, blockIdx.x, blockIdx.x == 0 && !ALONE ? ws.prefix : nullptr,
                                             seq, q0, nq);
    if (!any) {
        if (!ALONE) return;
        q0 = nq = 0;
    }
    float acc[R::N] = {}, z = 0.0f;
    for (int r = wave; r < nq; r += kLossWaves) {
        float l[R::N], p[R::N], soft[R::N], lse, top, inv;
        R::load(a.logits + (size_t)(q0 + r) * E, E, lane, l);
        probabilities<R::N, SIGMOID>(l, p, soft, lse, top, inv);
#pragma unroll
        for (int i = 0; i < R::N; ++i) acc[i] += p[i];
        z = fmaf(lse, lse, z);
    }
    const int32_t* ids = a.ids + (size_t)q0 * a.k;
    for (int i = threadIdx.x; i < nq * a.k; i += kLossThreads) {
        const int id = ids[i];
        if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
    }
#pragma unroll
    for (int i = 0; i < R::N; ++i) join[wave * R::N * 64 + R::element(i, lane)] = acc[i];
    z = group_sum<kLossWaves>(lane == 0 ? z : 0.0f);
    __syncthreads();
    const int e = threadIdx.x;
    float sum = 0.0f;
    if (e < E)
        for (int w = 0; w < kLossWaves; ++w) sum += join[w * R::N * 64 + e];
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

// Counts and means of 64 experts of a sequence: 64 columns by 16 lanes of parts.
__global__ __launch_bounds__(1024) void loss_join_kernel(const RouterArgs a, const LossParts ws) {
    __shared__ float sp[1024];
    __shared__ int sc[1024];
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
    if (lane > 0) return;
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
    if (threadIdx.x == 0) ws.balance[g * gridDim.y + blockIdx.y] = b;
}

__global__ __launch_bounds__(1024) void loss_sum_kernel(const RouterArgs a, const LossParts ws, int groups) {
    float b = 0.0f, z = 0.0f;
    for (int i = threadIdx.x; i < a.seqs.S * groups; i += 1024) b += ws.balance[i];
    const int parts = min(ws.prefix[a.seqs.S], ws.parts), n = rows_of_all(a.seqs);
    for (int i = threadIdx.x; i < parts; i += 1024) z += ws.z[i];
    b = group_sum<16>(b);
    z = group_sum<16>(z);
    if (threadIdx.x == 0) {
        a.losses[0] = n > 0 ? b * ((float)a.E / ((float)a.k * (float)n)) : 0.0f;
        a.losses[1] = n > 0 ? z / (float)n : 0.0f;
    }
}

// Rows of a part: 64 (four a wave) until there are 512 parts.
static int loss_rows(int T) {
    int per = 64;
    while ((long long)T / per > 512) per *= 2;
    return per;
}

static LossParts loss_parts(int T, int E, int G, void* ws, size_t* bytes) {
    LossParts l{};
    l.per = loss_rows(T);
    l.parts = T / l.per + (G < T ? G : T) + (T == 0);  // one at least: it writes the prefix
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
    if (bytes) *bytes = at;
    return l;
}

size_t balance_loss_workspace_bytes(int T, int E, int G) {
    size_t bytes = 0;
    loss_parts(T, E, G, nullptr, &bytes);
    return bytes;
}

template <int VEC, int NV>
static void launch_loss_rows(const RouterArgs& a, const LossParts& ws, bool alone, hipStream_t s) {
    const dim3 grid(alone ? 1 : ws.parts);
    if (a.score == MOE_SCORE_SIGMOID) {
        if (alone) loss_rows_kernel<VEC, NV, true, true><<<grid, kLossThreads, 0, s>>>(a, ws);
        else loss_rows_kernel<VEC, NV, true, false><<<grid, kLossThreads, 0, s>>>(a, ws);
    } else {
        if (alone) loss_rows_kernel<VEC, NV, false, true><<<grid, kLossThreads, 0, s>>>(a, ws);
        else loss_rows_kernel<VEC, NV, false, false><<<grid, kLossThreads, 0, s>>>(a, ws);
    }
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// launch<VEC, NV>() of the smallest row that holds E logits.
template <typename F>
static void by_width(int E, bool wide, F&& launch) {
    if (wide) {
        if (E <= 256) launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
        else if (E <= 512) launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
        else launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
    } else {
        if (E <= 64) launch(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
        else if (E <= 256) launch(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
        else launch(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
    }
}

hipError_t launch_balance_loss(const RouterArgs& a, hipStream_t s) {
    const int G = a.seqs.S, groups = (a.E + 63) / 64;
    const LossParts ws = loss_parts(a.T, a.E, G, a.ws, nullptr);
    const bool alone = G == 1 && a.T <= ws.per;
    by_width(a.E, a.E % 4 == 0 && aligned16(a.logits), [&](auto vec, auto nv) {
        launch_loss_rows<decltype(vec)::value, decltype(nv)::value>(a, ws, alone, s);
    });
    if (!alone) {
        loss_join_kernel<<<dim3(G, groups), 1024, 0, s>>>(a, ws);
        loss_sum_kernel<<<1, 1024, 0, s>>>(a, ws, groups);
    }
    return hipGetLastError();
}

// --------------------------------------------------------------- gradient

// Sequence of row t: the last one that begins at or before it, -1 if it lies in none.
__device__ __forceinline__ int sequence_of(const RowMap& m, int t, int lane) {
    if (!m.offsets) return 0;
    int before = 0;
    for (int s0 = 0; s0 <= m.S; s0 += 64) {
        const int s = s0 + lane;
        before += __popcll(__ballot(s <= m.S && m.offsets[min(s, m.S)] <= t));
    }
    return before >= 1 && before <= m.S ? before - 1 : -1;
}

// A wave a row.  Lane j < k holds pair j; the pairs' terms go to their logits' registers
// one by one.
template <int VEC, int NV, bool SIGMOID, int OUT>
__global__ __launch_bounds__(256) void route_grad_kernel(const RouterArgs a) {
    typedef Row<VEC, NV> R;
    const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), E = a.E;
    if (t >= a.T) return;
    const float* row = a.logits + (size_t)t * E;
    const int seq = a.counts ? sequence_of(a.seqs, t, lane) : -1;
    const bool whole = seq >= 0 || (a.dw && !SIGMOID && !a.renormalize);  // all logits count
    float d[R::N], p[R::N], soft[R::N], l[R::N], lse = 0.0f, top = 0.0f, inv = 0.0f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) d[i] = 0.0f;
    if (whole) {
        R::load(row, E, lane, l);
        probabilities<R::N, SIGMOID>(l, p, soft, lse, top, inv);
    }
    if (a.dw) {
        const int id = lane < a.k ? a.ids[(size_t)t * a.k + lane] : -1;
        const bool valid = id >= 0 && id < E;
        const float dw = valid ? a.scale * a.dw[(size_t)t * a.k + lane] : 0.0f, z = valid ? row[id] : -INFINITY;
        float term = 0.0f;  // the pair's own
        if (SIGMOID && !a.renormalize) {
            term = valid ? sigmoid_f32(z) * sigmoid_f32(-z) * dw : 0.0f;
        } else if (a.renormalize) {
            const float m = wave_max(z);
            float u = exp_f32(z - (m == -INFINITY ? 0.0f : m));
            if (SIGMOID) u = m < 0.0f ? u * sigmoid_f32(-z) : sigmoid_f32(z);
            const float sum = wave_sum(u);
            u = sum == 0.0f ? 0.0f : u / sum;
            const float dot = wave_sum(valid ? u * dw : 0.0f);
            term = valid ? u * (dw - dot) : 0.0f;
            if (SIGMOID) term = valid ? term * sigmoid_f32(-z) : 0.0f;
        } else {
            // softmax over all logits: the weights' sum pulls on every logit
            const float u = valid ? exp_f32(z - top) * inv : 0.0f;
            const float dot = wave_sum(valid ? u * dw : 0.0f);
            term = valid ? u * dw : 0.0f;
#pragma unroll
            for (int i = 0; i < R::N; ++i) d[i] = -soft[i] * dot;
        }
        for (int j = 0; j < a.k; ++j) {
            const int at = __builtin_amdgcn_readlane(id, j);
            const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(term), j));
            if (at < 0 || at >= E) continue;
            const int unit = at / VEC, reg = unit / 64 * VEC + at % VEC;
#pragma unroll
            for (int i = 0; i < R::N; ++i)
                if (i == reg) d[i] += lane == unit % 64 ? v : 0.0f;
        }
    }
    if (seq >= 0) {
        const float n = (float)rows_of_all(a.seqs), ng = (float)slot_range(a.seqs, seq).y;
        const float b = a.dlosses[0] * ((float)E / ((float)a.k * n)) / ng, zs = a.dlosses[1] * (2.0f / n) * lse;
        const int32_t* counts = a.counts + (size_t)seq * E;
        float f[R::N], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < R::N; ++i) {
            const int e = R::element(i, lane);
            f[i] = e < E ? b * (float)counts[e] : 0.0f;
            dot = fmaf(p[i], f[i], dot);
        }
        dot = wave_sum(dot);
#pragma unroll
        for (int i = 0; i < R::N; ++i) {
            float v = p[i] * (f[i] - dot);
            if (SIGMOID) v *= sigmoid_f32(-l[i]);
            d[i] += v + zs * soft[i];
        }
    }
    typedef typename DType<OUT>::type T;
    T* out = static_cast<T*>(a.dlogits) + (size_t)t * E;
#pragma unroll
    for (int g = 0; g < NV; ++g) {
        const int e = R::element(g * VEC, lane);
        if (e >= E) continue;
        if constexpr (VEC == 4) {
            typedef T t4 __attribute__((ext_vector_type(4)));
            t4 v;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = (T)d[4 * g + c];
            *reinterpret_cast<t4*>(out + e) = v;
        } else {
            out[e] = (T)d[g];
        }
    }
}

template <int VEC, int NV>
static void launch_route_grad(const RouterArgs& a, hipStream_t s) {
    const dim3 grid((a.T + 3) / 4);
    auto go = [&](auto sig, auto out) {
        route_grad_kernel<VEC, NV, decltype(sig)::value, decltype(out)::value><<<grid, 256, 0, s>>>(a);
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
    const bool wide = a.E % 4 == 0 && aligned16(a.logits) && aligned16(a.dlogits);
    by_width(a.E, wide, [&](auto vec, auto nv) { launch_route_grad<decltype(vec)::value, decltype(nv)::value>(a, s); });
    return hipGetLastError();
}

}  // namespace qmoe
