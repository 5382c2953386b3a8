// Expert products with few rows a slot: the weights are streamed once and
// every element goes from its load straight into a matrix instruction.
//
// Bound by HBM: a decode step reads each used matrix once (N K / 2 bytes of
// codes or 2 N K of 16-bit weights) for a handful of rows.  A workgroup owns
// 16 NT columns of one slot's product, its waves split K in segments of 256,
// and one LDS sum joins them: no second launch, no atomics, a fixed order.
//
// v_mfma_f32_16x16x32 takes the rows of x as its A operand (up to 16 a
// block, MB blocks) and 16 rows of w as its B operand: lane l holds eight
// inputs of weight row l % 16, which is what a 16-byte load along the row
// gives, so the weights pass through no LDS and need no shuffle.  Padding one
// row to 16 costs matrix-core time that a bandwidth-bound kernel has to
// spare, and spares the vector units the products, which for 4-bit weights
// they need for the dequantization.
//
// 4-bit weights: a byte 0..15 is the fp8 (e4m3) code of q / 512, so one
// v_cvt_scalef32_pk_{bf16,f16}_fp8 with scale 512 turns two codes into two
// exact 16-bit values: 7 instructions for 8 weights.  It yields elements
// 0 2 4 6 1 3 5 7 of a word; the x fragments are put in that order (four byte
// permutes for 16 rows x 8 inputs), the sum does not care.  With zero points
//   sum_j s (q_j - z) x_j = s (sum_j q_j x_j - z sum_j x_j),
// where sum_j x_j comes from one more matrix instruction against ones, in
// the accumulator's own layout.  PER matrix instructions (32 inputs each)
// share a group; groups of less than 128 inputs need each instruction's 32
// inputs from one run, which a 4 x 4 transposition of words between the
// lanes' quarters gives (v_permlane16/32_swap).
#pragma once
#include <type_traits>

#include "expert_ops.h"

namespace qmoe {

struct StreamArgs {
    const void* x;
    const void* w;      // 16-bit weights or code bytes
    size_t w_stride;    // bytes from slot to slot
    const void* scales;
    const uint8_t* zeros;
    int scale_f32, group_shift;
    int N, K;
    RowMap rows;
    int x_rows, y_rows;
    void* y;
    int y_f32;
};

constexpr int kSegment = 256;  // inputs a wave takes at a time
// Waves that split a workgroup's inputs.  Four: more would leave a CU one or
// two workgroups (128 experts of 4096 x 7168 at 12 rows a slot takes 671
// us, with eight 792 us).
constexpr int kStreamWaves = 4;

template <int DT>
__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
    if constexpr (DT == MOE_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
}

// Eight codes of a word -> elements 0 2 4 6 1 3 5 7 as exact 16-bit values.
template <int DT>
__device__ __forceinline__ uint4 codes_frag(uint32_t w) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    uint4 f;
    if constexpr (DT == MOE_BF16) {
        f.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
        f.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
        f.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
        f.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
    } else {
        f.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false));
        f.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true));
        f.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false));
        f.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true));
    }
    return f;
}

// Eight 16-bit values in the order of codes_frag.
__device__ __forceinline__ uint4 codes_order(uint4 v) {
    return make_uint4(__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                      __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u));
}

// Word j of lane quarter c <- word c of quarter j (quarter = lane / 16).
__device__ __forceinline__ uint4 transpose_quarters(uint4 v) {
    const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return make_uint4(c[0], c[1], d[0], d[1]);
}

// An unaligned load.
template <typename T>
__device__ __forceinline__ T load_bytes(const uint8_t* p) {
    T v;
    __builtin_memcpy(&v, p, sizeof v);
    return v;
}

// The value that the first quarter's lane of the same lane % 16 holds.
__device__ __forceinline__ uint32_t first_quarter(uint32_t v) {
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false)[0];
}

// Slot of index i: with fewer positions than slots the i-th slot that owns
// one (found by a ballot scan), otherwise slot i.  -1: none.
__device__ __forceinline__ int stream_slot(const RowMap& m, int i) {
    if (!m.offsets || m.R >= m.S) return i;
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int s0 = 0; s0 < m.S; s0 += 256) {
        bool owns[4];  // four loads in flight, then the ballots
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = s0 + 64 * j + lane;
            owns[j] = slot_range(m, min(s, m.S - 1)).y > 0 && s < m.S;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint64_t mask = __ballot(owns[j]);
            const int n = __popcll(mask);
            if (i < before + n) {
                for (int k = i - before; k > 0; --k) mask &= mask - 1;
                return s0 + 64 * j + __ffsll((unsigned long long)mask) - 1;
            }
            before += n;
        }
    }
    return -1;
}

// WT 0: 16-bit weights, 1: 4-bit.  SWI: tile 0 holds gate rows, tile 1 the up
// rows of the same 16 features (NT = 2).
template <int WT, int DT, int NT, int MB, int PER, bool SWI>
__global__ __launch_bounds__(64 * kStreamWaves) void expert_stream_kernel(const StreamArgs a) {
    typedef typename DType<DT>::type E;
    extern __shared__ float red[];  // [waves][NT][MB][64][4]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int col = lane & 15, c = lane >> 4;
    const int slot = __builtin_amdgcn_readfirstlane(stream_slot(a.rows, blockIdx.y));
    if (slot < 0) return;
    const int2 r = slot_range(a.rows, slot);
    const int N = a.N, K = a.K, half = N / 2, width = SWI ? half : N;
    const int n0 = blockIdx.x * (SWI ? 16 : 16 * NT);
    const uint8_t* w = static_cast<const uint8_t*>(a.w) + (size_t)slot * a.w_stride;
    const uint8_t* wp[NT];
    size_t sp[NT];  // first scale of the lane's weight row
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = SWI ? min(n0 + col, half - 1) + t * half : min(n0 + 16 * t + col, N - 1);
        wp[t] = w + (WT ? (size_t)n * (K / 2) : (size_t)n * K * 2);
        sp[t] = WT ? ((size_t)slot * N + n) * (K >> a.group_shift) : 0;
    }
    for (int rb = 0; rb < r.y; rb += 16 * MB) {
        const int nr = min(r.y - rb, 16 * MB);
        // The lane's x rows: requested first, turned into addresses only behind
        // the first weight loads, so that those do not wait for them.
        int xrow[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) xrow[m] = pair_of(a.rows, a.x_rows, r.x + rb + min(16 * m + col, nr - 1));
        f32x4 tot[NT][MB] = {};
        // A segment of 256 inputs: its weights, scales and zeros as loaded.
        constexpr int LD = WT ? 2 : 8;        // 16-byte weight loads a tile
        constexpr int SG = WT ? 8 / PER : 2;  // groups of the segment
        constexpr int XI = MB == 4 ? 4 : 8;   // x instructions held at a time: 64 rows of eight would spill
        typedef uint32_t s16v __attribute__((ext_vector_type(SG / 2)));
        typedef uint32_t s32v __attribute__((ext_vector_type(SG)));
        auto run = [&](auto scale_tag, auto zero_tag) {
            constexpr bool SCALE_F32 = decltype(scale_tag)::value, ZEROS = decltype(zero_tag)::value;
            struct Segment {
                uint4 w[NT][LD];
                s16v s16[NT];
                s32v s32[NT];
                uint64_t z[NT];
            };
            // CUT: the row's last segment, shorter than 256
            auto load = [&](Segment& v, int k0, auto cut_tag) {
                constexpr bool CUT = decltype(cut_tag)::value;
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int k = WT ? k0 + 128 * i + 32 * c : k0 + 32 * i + 8 * c;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (CUT) v.w[t][i] = make_uint4(0, 0, 0, 0);
                        if (!CUT || k < K) v.w[t][i] = *reinterpret_cast<const uint4*>(wp[t] + (WT ? k / 2 : k * 2));
                    }
                }
                if constexpr (WT) {
                    // A row's groups of the segment lie side by side: one load of
                    // up to 16 bytes (2- or 1-byte aligned), since single values
                    // cost the address unit a lane at a time.
                    // The four quarters want the same values: the first loads them.
                    auto at = [&](int t, int g) { return sp[t] + (min(k0 + 32 * PER * g, K - 1) >> a.group_shift); };
                    if (CUT || c == 0)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if constexpr (SCALE_F32) {
                            const uint32_t* p = static_cast<const uint32_t*>(a.scales);
                            if (!CUT) __builtin_memcpy(&v.s32[t], p + at(t, 0), 4 * SG);
                            else
#pragma unroll
                                for (int g = 0; g < SG; ++g) v.s32[t][g] = p[at(t, g)];
                        } else {
                            const uint16_t* p = static_cast<const uint16_t*>(a.scales);
                            if (!CUT) __builtin_memcpy(&v.s16[t], p + at(t, 0), 2 * SG);
                            else
#pragma unroll
                                for (int g = 0; g < SG; g += 2) v.s16[t][g / 2] = p[at(t, g)] | (uint32_t)p[at(t, g + 1)] << 16;
                        }
                        if constexpr (ZEROS) {
                            v.z[t] = 0;
                            if (!CUT) {
                                if constexpr (SG == 2) v.z[t] = load_bytes<uint16_t>(a.zeros + at(t, 0));
                                else if constexpr (SG == 4) v.z[t] = load_bytes<uint32_t>(a.zeros + at(t, 0));
                                else v.z[t] = load_bytes<uint64_t>(a.zeros + at(t, 0));
                            } else
#pragma unroll
                                for (int g = 0; g < SG; ++g) v.z[t] |= (uint64_t)a.zeros[at(t, g)] << (8 * g);
                        }
                    }
                }
            };
            uint4 xv[MB][XI];
            // x fragments: instruction i takes the inputs that the weights'
            // words hold; lanes of rows past the batch load nothing
            auto load_x = [&](int k0, int i0, auto cut_tag) {
                constexpr bool CUT = decltype(cut_tag)::value;
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    if (CUT)
#pragma unroll
                        for (int j = 0; j < XI; ++j) xv[m][j] = make_uint4(0, 0, 0, 0);
                    int row = xrow[m];
                    asm("" : "+v"(row));  // not hoisted above the weight loads
                    const E* xp = static_cast<const E*>(a.x) + (size_t)row_of_pair(a.rows, a.x_rows, row) * K;
                    if (16 * m + col < nr) {
#pragma unroll
                        for (int j = 0; j < XI; ++j) {
                            const int i = i0 + j;
                            const int k = WT && PER == 4 ? k0 + 128 * (i / 4) + 32 * c + 8 * (i % 4) : k0 + 32 * i + 8 * c;
                            if (!CUT || k < K) xv[m][j] = *reinterpret_cast<const uint4*>(xp + k);
                        }
                    }
                }
            };
            // what stands between a segment's loads and its use
            auto arrange = [&](Segment& v, auto cut_tag) {
                if constexpr (WT && !decltype(cut_tag)::value) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if constexpr (SCALE_F32) {
#pragma unroll
                            for (int g = 0; g < SG; ++g) v.s32[t][g] = first_quarter(v.s32[t][g]);
                        } else {
#pragma unroll
                            for (int g = 0; g < SG / 2; ++g) v.s16[t][g] = first_quarter(v.s16[t][g]);
                        }
                        if constexpr (ZEROS) {
                            const uint32_t lo = first_quarter((uint32_t)v.z[t]);
                            const uint32_t hi = SG > 4 ? first_quarter((uint32_t)(v.z[t] >> 32)) : 0u;
                            v.z[t] = (uint64_t)hi << 32 | lo;
                        }
                    }
                }
                if constexpr (WT && PER < 4) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < LD; ++i) v.w[t][i] = transpose_quarters(v.w[t][i]);
                }
            };
            // x instructions i0 .. i0 + XI of a segment
            auto multiply = [&](const Segment& v, int k0, int i0, auto cut_tag) {
                constexpr bool CUT = decltype(cut_tag)::value;
                if constexpr (WT) {
                    const uint32_t one = DT == MOE_BF16 ? 0x3F803F80u : 0x3C003C00u;
                    const uint4 ones = make_uint4(one, one, one, one);
#pragma unroll
                    for (int m = 0; m < MB; ++m)
#pragma unroll
                        for (int j = 0; j < XI; ++j) xv[m][j] = codes_order(xv[m][j]);
#pragma unroll
                    for (int g = i0 / PER; g < (i0 + XI) / PER; ++g) {
                        f32x4 acc[NT][MB] = {}, sx[MB] = {};
#pragma unroll
                        for (int p = 0; p < PER; ++p) {
                            const int i = g * PER + p;
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const uint4 u = v.w[t][i / 4];
                                const uint4 f = codes_frag<DT>(i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w);
#pragma unroll
                                for (int m = 0; m < MB; ++m) acc[t][m] = mfma16<DT>(xv[m][i - i0], f, acc[t][m]);
                            }
#pragma unroll
                            for (int m = 0; m < MB; ++m) sx[m] = mfma16<DT>(xv[m][i - i0], ones, sx[m]);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float sc;
                            if constexpr (SCALE_F32) {
                                sc = __uint_as_float(v.s32[t][g]);
                            } else {
                                const uint32_t h = v.s16[t][g / 2] >> (16 * (g & 1)) & 0xFFFFu;
                                sc = DT == MOE_BF16 ? __uint_as_float(h << 16)
                                                    : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
                            }
                            if (CUT && k0 + 32 * PER * g >= K) sc = 0.0f;
                            const float z = ZEROS ? (float)((uint32_t)(v.z[t] >> (8 * g)) & 0xFFu) : 8.0f;
#pragma unroll
                            for (int m = 0; m < MB; ++m)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    tot[t][m][e] = fmaf(sc, fmaf(-z, sx[m][e], acc[t][m][e]), tot[t][m][e]);
                        }
                        if (MB == 4) __builtin_amdgcn_sched_barrier(0);  // a group at a time: hoisted fragments spill
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < XI; ++j)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int m = 0; m < MB; ++m) tot[t][m] = mfma16<DT>(xv[m][j], v.w[t][i0 + j], tot[t][m]);
                }
            };
            const int step = waves * kSegment;
            int k0 = wave * kSegment;
            // (Loading the next segment while this one multiplies costs a quarter
            // of the waves their registers and gains nothing.)
            for (; k0 + kSegment <= K; k0 += step) {
                Segment now;
                load(now, k0, std::false_type{});
                load_x(k0, 0, std::false_type{});
                arrange(now, std::false_type{});
#pragma unroll
                for (int i0 = 0; i0 < 8; i0 += XI) {
                    if (i0) load_x(k0, i0, std::false_type{});
                    multiply(now, k0, i0, std::false_type{});
                }
            }
            if (k0 < K) {
                Segment now;
                load(now, k0, std::true_type{});
                load_x(k0, 0, std::true_type{});
                arrange(now, std::true_type{});
#pragma unroll
                for (int i0 = 0; i0 < 8; i0 += XI) {
                    if (i0) load_x(k0, i0, std::true_type{});
                    multiply(now, k0, i0, std::true_type{});
                }
            }
        };
        // one loop for each kind of scales and zeros: a branch on them between
        // the loads costs a wait for what is in flight
        if (WT && a.scale_f32 && a.zeros) run(std::true_type{}, std::true_type{});
        else if (WT && a.scale_f32) run(std::true_type{}, std::false_type{});
        else if (WT && a.zeros) run(std::false_type{}, std::true_type{});
        else run(std::false_type{}, std::false_type{});
        // join the waves' parts in wave order; element (row, col) of a block
        // sits at lane 16 (row / 4) + col, component row % 4
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < MB; ++m)
                *reinterpret_cast<f32x4*>(red + (((wave * NT + t) * MB + m) * 64 + lane) * 4) = tot[t][m];
        __syncthreads();
        constexpr int TILES = SWI ? 1 : NT;
        for (int o = threadIdx.x; o < TILES * nr * 16; o += blockDim.x) {
            const int cc = o & 15, row = (o >> 4) % nr, t = (o >> 4) / nr;
            const int at = ((row >> 4) * 64 + ((row & 15) >> 2) * 16 + cc) * 4 + (row & 3);
            float v[2] = {0.0f, 0.0f};
            for (int u = 0; u < waves; ++u) {
                v[0] += red[(u * NT + t) * MB * 256 + at];
                if (SWI) v[1] += red[(u * NT + 1) * MB * 256 + at];
            }
            const int n = n0 + 16 * t + cc;
            if (n >= width) continue;
            if (SWI) v[0] = v[0] * sigmoid_f32(v[0]) * v[1];
            const size_t out = (size_t)row_of(a.rows, a.y_rows, r.x + rb + row) * width + n;
            if (a.y_f32) static_cast<float*>(a.y)[out] = v[0];
            else static_cast<E*>(a.y)[out] = (E)v[0];
        }
        __syncthreads();
    }
}

template <int WT, int DT, int NT, int PER, bool SWI>
static hipError_t stream_launch_rows(const StreamArgs& a, int mb, dim3 grid, int waves, hipStream_t s) {
    const size_t lds = (size_t)waves * NT * mb * 1024;
    if (mb == 1) expert_stream_kernel<WT, DT, NT, 1, PER, SWI><<<grid, 64 * waves, lds, s>>>(a);
    else if (mb == 2 || PER == 1) expert_stream_kernel<WT, DT, NT, 2, PER, SWI><<<grid, 64 * waves, lds, s>>>(a);
    else if constexpr (PER > 1) expert_stream_kernel<WT, DT, NT, 4, PER, SWI><<<grid, 64 * waves, lds, s>>>(a);
    return hipGetLastError();
}

template <int WT, int DT, int PER>
static hipError_t stream_launch(const StreamArgs& a, int act, hipStream_t s) {
    if (a.rows.R == 0) return hipSuccess;
    const int slots = a.rows.offsets ? (a.rows.R < a.rows.S ? a.rows.R : a.rows.S) : 1;
    const int mean = (a.rows.R + slots - 1) / slots;
    // Rows a pass: twice the mean and more, so that a slot above it still
    // takes one pass over its weights; 64 rows of groups of 32 would spill.
    const int mb = mean <= 8 || a.rows.R <= 16 ? 1 : mean <= 16 || a.rows.R <= 32 || PER == 1 ? 2 : 4;
    const int segs = (a.K + kSegment - 1) / kSegment, turns = (segs + kStreamWaves - 1) / kStreamWaves;
    const int waves = (segs + turns - 1) / turns;
    const int width = act ? a.N / 2 : a.N;
    if (act) return stream_launch_rows<WT, DT, 2, PER, true>(a, mb, dim3((width + 15) / 16, slots), waves, s);
    const int tiles = (width + 15) / 16;
    // one tile a workgroup while that leaves CUs without one
    if ((long long)tiles * slots <= 512)
        return stream_launch_rows<WT, DT, 1, PER, false>(a, mb, dim3(tiles, slots), waves, s);
    return stream_launch_rows<WT, DT, 2, PER, false>(a, mb, dim3((tiles + 1) / 2, slots), waves, s);
}

template <int DT>
static hipError_t stream_launch_type(const StreamArgs& a, int w4, int act, hipStream_t s) {
    if (!w4) return stream_launch<0, DT, 4>(a, act, s);
    switch (a.group_shift) {
        case 5: return stream_launch<1, DT, 1>(a, act, s);
        case 6: return stream_launch<1, DT, 2>(a, act, s);
        default: return stream_launch<1, DT, 4>(a, act, s);
    }
}

hipError_t launch_stream_bf16(const StreamArgs& a, int w4, int act, hipStream_t s);
hipError_t launch_stream_f16(const StreamArgs& a, int w4, int act, hipStream_t s);

}  // namespace qmoe
