// Expert products with few rows a slot: the weights are streamed once and
// every element goes from its load straight into a matrix instruction.
//
// Bound by HBM: a decode step reads each used matrix once (N K / 2 bytes of
// codes or 2 N K of 16-bit weights) for a handful of rows.  A workgroup owns
// 16 NT columns of one slot's product, its waves split K in segments of 256,
// and one LDS sum joins them: no second launch, no atomics, a fixed order.
// Measured for 16 experts of 1536 x 2048 with SwiGLU, a row each: bf16 20 us
// (5.0 TB/s), 4-bit in groups of 64 9.4 us.
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
// v_cvt_scalef32_pk_{bf16,f16}_fp8 scaled by 512 (and by kCodeUnit) turns two codes
// into two exact 16-bit values: 7 instructions for 8 weights.  It yields elements
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

#include "act.h"
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
    int slots;       // slots that can own a position
    int unit_shift;  // a workgroup walks up to 2^unit_shift rows of a slot
    Epilogue epi;    // biased products
};

constexpr int kSegment = 256;  // inputs a wave takes at a time
// Groups of a row whose scales and zeros the workgroup holds in LDS (loaded by
// the waves for each segment, a few bytes of 16 rows at a time, they took 13 %
// of a pool's time).  The stride puts 16 rows on different banks.
constexpr int kTableGroups = 64, kTableStride = kTableGroups + 2;
// Rows up to which 4-bit products share out the loads of x.  With the table,
// 192 experts of 4096 x 7168 for 256 pairs: 711 -> 521 us, 5.7 TB/s of codes,
// scales and zeros.  (16-bit weights have four times the bytes a load of x:
// no gain.)
constexpr int kFewRows = 4;
// Waves that split a workgroup's inputs.  Four: more would leave a CU one or
// two workgroups (128 4-bit experts of 4096 x 7168 take 353 us at 1.5 rows a
// slot and 1044 us at 30, with eight 420 and 1229 us).  With few workgroups, by
// four and by eight: one bf16 matrix of 2048 x 2048 5.0 and 5.0 us (128
// workgroups), one 4-bit matrix of 4096 x 2048 4.2 and 4.2, of 4096 x 4096 6.4 and
// 5.7 (256), 16 4-bit gate/up of 1536 x 2048 8.7 and 10.8 (768).
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

// What the codes and the ones against which x is summed are multiplied by: a
// group's sums of code x and zero x reach 2^15 x, which for bf16 x near its
// largest would overflow although scale (code - zero) x does not.  All of a row's
// sums carry the factor, exactly but below 2^-110; the store takes it out.  fp16 x
// has no such values.
template <int DT> constexpr float kCodeUnit = DT == MOE_BF16 ? 1.0f / 65536.0f : 1.0f;

// Eight codes of a word -> elements 0 2 4 6 1 3 5 7 as exact 16-bit values, times
// kCodeUnit.
template <int DT>
__device__ __forceinline__ uint4 codes_frag(uint32_t w) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    constexpr float unit = 512.0f * kCodeUnit<DT>;
    uint4 f;
    if constexpr (DT == MOE_BF16) {
        f.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, unit, false));
        f.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, unit, true));
        f.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, unit, false));
        f.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, unit, true));
    } else {
        f.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, unit, false));
        f.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, unit, true));
        f.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, unit, false));
        f.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, unit, true));
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

// Lane l of a row of 16 <- lane l + N.
template <int N>
__device__ __forceinline__ uint4 row_shift(uint4 v) {
    auto one = [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x100 + N, 0xF, 0xF, true); };
    return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
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

// Of the units of 2^shift rows behind the first of each slot, in slot order, number
// e: its slot (-1: there are fewer) and first row.  A scan over the slots (S <=
// 1024) in each wave: a lane counts up to 16 neighbouring slots.
__device__ __forceinline__ int2 later_unit(const RowMap& m, int e, int shift) {
    if (!m.offsets) return make_int2((m.R - 1) >> shift > e ? 0 : -1, (e + 1) << shift);
    const int lane = threadIdx.x & 63, per = (m.S + 63) / 64, s0 = lane * per;
    int n[16], mine = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) n[j] = j < per && s0 + j < m.S ? max(slot_range(m, s0 + j).y - 1, 0) >> shift : 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) mine += n[j];
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(sum, o, 64);
        if (lane >= o) sum += x;
    }
    const uint64_t mask = __ballot(e < sum);
    if (!mask) return make_int2(-1, 0);
    int slot = -1, unit = 0, left = e - (sum - mine);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        if (slot < 0 && left < n[j]) slot = s0 + j, unit = left + 1;
        left -= n[j];
    }
    const int from = __ffsll((unsigned long long)mask) - 1;
    return make_int2(__builtin_amdgcn_readlane(slot, from), __builtin_amdgcn_readlane(unit, from) << shift);
}

// The launch bounds' second number keeps the sums in ordinary registers: the
// accumulation registers would be read back one by one for the scales.
// WT 0: 16-bit weights, 1: 4-bit.  SWI: tile 0 holds gate rows, tile 1 the up
// rows of the same 16 features (NT = 2).  EPI: the store adds bias and residual.
template <int WT, int DT, int NT, int MB, int PER, bool SWI, bool EPI>
__global__ __launch_bounds__(64 * kStreamWaves, MB == 4 ? 1 : WT && MB == 1 ? 4 : 2) void expert_stream_kernel(const StreamArgs a) {
    typedef typename DType<DT>::type E;
    extern __shared__ float red[];  // [waves][NT][MB][64][4]; before that the table of scales
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int col = lane & 15, c = lane >> 4;
    // The first units of all slots, then the later ones.
    int2 begin;
    if ((int)blockIdx.y < a.slots) begin = make_int2(stream_slot(a.rows, blockIdx.y), 0);
    else begin = later_unit(a.rows, blockIdx.y - a.slots, a.unit_shift);
    const int slot = __builtin_amdgcn_readfirstlane(begin.x), rb0 = __builtin_amdgcn_readfirstlane(begin.y);
    if (slot < 0) return;
    int2 r = slot_range(a.rows, slot);
    r.y = min(r.y, rb0 + (1 << a.unit_shift));
    const int N = a.N, K = a.K, half = N / 2, width = SWI ? half : N;
    const int n0 = blockIdx.x * (SWI ? 16 : 16 * NT);
    const uint8_t* w = static_cast<const uint8_t*>(a.w) + (size_t)slot * a.w_stride;
    const uint8_t* wp[NT];
    auto weight_row = [&](int row) {  // of the workgroup's 16 NT
        return SWI ? min(n0 + row % 16, half - 1) + row / 16 * half : min(n0 + row, N - 1);
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) wp[t] = w + (size_t)weight_row(16 * t + col) * (WT ? K / 2 : K * 2);
    // Scales and zeros of groups g0 to g0 + kTableGroups of the workgroup's
    // rows, as fp32 pairs; a zero scale behind a row's end.
    float2* table = reinterpret_cast<float2*>(red);
    auto fill = [&](int g0) {
        const int groups = K >> a.group_shift;
        for (int u = threadIdx.x; u < 2 * NT * kTableGroups; u += blockDim.x) {
            const int row = u / (kTableGroups / 8), at = u % (kTableGroups / 8) * 8, left = groups - g0 - at;
            if (left <= 0) continue;
            const size_t from = ((size_t)slot * N + weight_row(row)) * groups + g0 + at;
            float2 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = make_float2(0.0f, 8.0f);
            if (left >= 8) {
                uint64_t z = 0;
                if (a.zeros) z = load_bytes<uint64_t>(a.zeros + from);
                if (a.scale_f32) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i].x = static_cast<const float*>(a.scales)[from + i];
                } else {
                    const uint4 v = load_bytes<uint4>(static_cast<const uint8_t*>(a.scales) + from * 2);
                    const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        q[i].x = (float)__builtin_bit_cast(E, (uint16_t)(h[i / 2] >> (16 * (i & 1))));
                }
                if (a.zeros)
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i].y = (float)((uint32_t)(z >> (8 * i)) & 0xFFu);
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i) {
                    if (i >= left) continue;
                    q[i].x = a.scale_f32 ? static_cast<const float*>(a.scales)[from + i]
                                         : (float)static_cast<const E*>(a.scales)[from + i];
                    if (a.zeros) q[i].y = (float)a.zeros[from + i];
                }
            }
            float4* to = reinterpret_cast<float4*>(table + row * kTableStride + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = make_float4(q[2 * i].x, q[2 * i].y, q[2 * i + 1].x, q[2 * i + 1].y);
        }
    };
    for (int rb = rb0; rb < r.y; rb += 16 * MB) {
        const int nr = min(r.y - rb, 16 * MB);
        f32x4 tot[NT][MB] = {};
        // A pass over the weights.  XR: rows that share one load of x.
        auto pass = [&](auto xr_tag) {
            constexpr int XR = decltype(xr_tag)::value;
            constexpr bool FEW = XR == kFewRows;
            constexpr int LD = WT ? 2 : 8;         // 16-byte weight loads a tile
            constexpr int XI = MB == 4 ? 4 : 8;    // x instructions held at a time: 64 rows of eight would spill
            constexpr int XL = FEW ? XR / 2 : XI;  // x loads of those
            // The lane's x rows: requested first, turned into addresses only behind
            // the first weight loads, so that those do not wait for them.
            int xrow[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m)
                xrow[m] = pair_of(a.rows, a.x_rows, r.x + rb + min(16 * m + (FEW ? col % XR : col), nr - 1));
            typedef uint4 Weights[NT][LD];
            typedef uint4 Xv[MB][XL];
            // CUT: the row's last segment, shorter than 256
            auto load = [&](Weights& v, int k0, auto cut_tag) {
                constexpr bool CUT = decltype(cut_tag)::value;
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int k = WT ? k0 + 128 * i + 32 * c : k0 + 32 * i + 8 * c;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (CUT) v[t][i] = make_uint4(0, 0, 0, 0);
                        if (!CUT || k < K) v[t][i] = *reinterpret_cast<const uint4*>(wp[t] + (WT ? k / 2 : k * 2));
                    }
                }
            };
            // x fragments: instruction i takes the inputs that the weights' words
            // hold; lanes of rows past the batch load nothing (their rows of
            // the sums are not stored).  Up to four rows: the lanes that have no
            // row bring other instructions' inputs (lane col: row col % 4,
            // instruction 4 j + col / 4), two loads a segment instead of eight of
            // the same cost.
            auto load_x = [&](Xv& xv, int k0, int i0, auto cut_tag) {
                constexpr bool CUT = decltype(cut_tag)::value;
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    if (CUT)
#pragma unroll
                        for (int j = 0; j < XL; ++j) xv[m][j] = make_uint4(0, 0, 0, 0);
                    int row = xrow[m];
                    asm("" : "+v"(row));  // not hoisted above the weight loads
                    const E* xp = static_cast<const E*>(a.x) + (size_t)row_of_pair(a.rows, a.x_rows, row) * K;
                    if (FEW || 16 * m + col < nr) {
#pragma unroll
                        for (int j = 0; j < XL; ++j) {
                            const int i = FEW ? 16 / XR * j + col / XR : i0 + j;
                            const int k = WT && PER == 4 ? k0 + 128 * (i / 4) + 32 * c + 8 * (i % 4) : k0 + 32 * i + 8 * c;
                            if (!CUT || k < K) xv[m][j] = *reinterpret_cast<const uint4*>(xp + k);
                        }
                    }
                }
            };
            auto fragment = [&](const Xv& xv, int m, int i) {  // of instruction i (of those held)
                if constexpr (FEW) {
                    const uint4 v = xv[m][i / 4];
                    return i % 4 == 0 ? v : i % 4 == 1 ? row_shift<4>(v) : i % 4 == 2 ? row_shift<8>(v) : row_shift<12>(v);
                } else {
                    return xv[m][i];
                }
            };
            // x instructions i0 .. i0 + XI of a segment
            auto multiply = [&](const Weights& v, Xv& xv, int k0, int i0, int c0) {
                if constexpr (WT) {
                    const uint32_t one = DT == MOE_BF16 ? 0x37803780u : 0x3C003C00u;  // kCodeUnit twice
                    const uint4 ones = make_uint4(one, one, one, one);
                    const int g0 = (k0 - c0) >> a.group_shift;
#pragma unroll
                    for (int m = 0; m < MB; ++m)
#pragma unroll
                        for (int j = 0; j < XL; ++j) xv[m][j] = codes_order(xv[m][j]);
#pragma unroll
                    for (int g = i0 / PER; g < (i0 + XI) / PER; ++g) {
                        f32x4 acc[NT][MB] = {}, sx[MB] = {};
#pragma unroll
                        for (int p = 0; p < PER; ++p) {
                            const int i = g * PER + p;
                            uint4 xf[MB];
#pragma unroll
                            for (int m = 0; m < MB; ++m) xf[m] = fragment(xv, m, i - i0);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const uint4 u = v[t][i / 4];
                                const uint4 f = codes_frag<DT>(i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w);
#pragma unroll
                                for (int m = 0; m < MB; ++m) acc[t][m] = mfma16<DT>(xf[m], f, acc[t][m]);
                            }
#pragma unroll
                            for (int m = 0; m < MB; ++m) sx[m] = mfma16<DT>(xf[m], ones, sx[m]);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float2 q = table[(16 * t + col) * kTableStride + g0 + g];
#pragma unroll
                            for (int m = 0; m < MB; ++m)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    tot[t][m][e] = fmaf(q.x, fmaf(-q.y, sx[m][e], acc[t][m][e]), tot[t][m][e]);
                        }
                        __builtin_amdgcn_sched_barrier(0);  // a group at a time: hoisted fragments spill
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < XI; ++j) {
                        uint4 xf[MB];
#pragma unroll
                        for (int m = 0; m < MB; ++m) xf[m] = fragment(xv, m, j);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int m = 0; m < MB; ++m) tot[t][m] = mfma16<DT>(xf[m], v[t][i0 + j], tot[t][m]);
                    }
                }
            };
            auto segment = [&](Weights& v, Xv& xv, int k0, int c0, auto cut_tag) {
                if constexpr (WT && PER < 4) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < LD; ++i) v[t][i] = transpose_quarters(v[t][i]);
                }
#pragma unroll
                for (int i0 = 0; i0 < 8; i0 += XI) {
                    if (i0) load_x(xv, k0, i0, cut_tag);
                    multiply(v, xv, k0, i0, c0);
                }
            };
            const std::false_type whole;
            const std::true_type cut;
            const int step = waves * kSegment, span = WT ? kTableGroups << a.group_shift : K;
            int k0 = wave * kSegment, c0 = 0;
            while (true) {
                if (WT) {
                    fill(c0 >> a.group_shift);
                    __syncthreads();
                }
                for (; k0 + kSegment <= K && k0 - c0 < span; k0 += step) {
                    Weights now;
                    Xv xv;
                    load(now, k0, whole);
                    load_x(xv, k0, 0, whole);
                    segment(now, xv, k0, c0, whole);
                }
                if (!WT || K - c0 <= span) break;
                c0 += span;
                __syncthreads();
            }
            if (k0 < K) {
                Weights now;
                Xv xv;
                load(now, k0, cut);
                load_x(xv, k0, 0, cut);
                segment(now, xv, k0, c0, cut);
            }
        };
        if constexpr (WT && MB == 1) {
            if (nr <= kFewRows) pass(std::integral_constant<int, kFewRows>{});
            else pass(std::integral_constant<int, 16>{});
        } else {
            pass(std::integral_constant<int, 16>{});
        }
        if (WT) __syncthreads();  // the sums take the table's place
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
            if (WT) v[0] *= 1.0f / kCodeUnit<DT>, v[1] *= 1.0f / kCodeUnit<DT>;
            const size_t yrow = (size_t)row_of(a.rows, a.y_rows, r.x + rb + row), out = yrow * width + n;
            if constexpr (EPI) {
                const size_t at = (size_t)slot * N + n, zat = yrow * N + n;
                if (a.epi.bias) {
                    v[0] += a.epi.bias_f32 ? static_cast<const float*>(a.epi.bias)[at] : (float)static_cast<const E*>(a.epi.bias)[at];
                    if (SWI) v[1] += a.epi.bias_f32 ? static_cast<const float*>(a.epi.bias)[at + half]
                                                    : (float)static_cast<const E*>(a.epi.bias)[at + half];
                }
                if (a.epi.z) {
                    static_cast<E*>(a.epi.z)[zat] = (E)v[0];
                    if (SWI) static_cast<E*>(a.epi.z)[zat + half] = (E)v[1];
                }
                if (!SWI) v[0] = act1(a.epi.act, v[0]);
            }
            if (SWI) v[0] = v[0] * sigmoid_f32(v[0]) * v[1];
            if constexpr (EPI) {
                if (a.epi.residual)
                    v[0] += a.epi.res_f32 ? static_cast<const float*>(a.epi.residual)[out]
                                          : (float)static_cast<const E*>(a.epi.residual)[out];
            }
            if (a.y_f32) static_cast<float*>(a.y)[out] = v[0];
            else static_cast<E*>(a.y)[out] = (E)v[0];
        }
        __syncthreads();
    }
}

template <int WT, int DT, int NT, int PER, bool SWI, bool EPI>
static hipError_t stream_launch_rows(const StreamArgs& a, int mb, dim3 grid, int waves, hipStream_t s) {
    const size_t sums = (size_t)waves * NT * mb * 1024, table = WT ? 16 * NT * kTableStride * sizeof(float2) : 0;
    const size_t lds = sums > table ? sums : table;
    if (mb == 1) expert_stream_kernel<WT, DT, NT, 1, PER, SWI, EPI><<<grid, 64 * waves, lds, s>>>(a);
    else if (mb == 2) expert_stream_kernel<WT, DT, NT, 2, PER, SWI, EPI><<<grid, 64 * waves, lds, s>>>(a);
    else if constexpr (PER > 1 && (NT == 1 || SWI)) expert_stream_kernel<WT, DT, NT, 4, PER, SWI, EPI><<<grid, 64 * waves, lds, s>>>(a);
    return hipGetLastError();
}

template <int WT, int DT, int PER, bool EPI = false>
static hipError_t stream_launch(const StreamArgs& a, int act, hipStream_t s) {
    if (a.rows.R == 0) return hipSuccess;
    const int slots = a.rows.offsets ? (a.rows.R < a.rows.S ? a.rows.R : a.rows.S) : 1;
    const int mean = (a.rows.R + slots - 1) / slots;
    const int width = act ? a.N / 2 : a.N, tiles = (width + 15) / 16;
    const bool few = (long long)tiles * slots <= 512;
    // Blocks of 16 rows a pass.  Fewer leave the CUs more waves, and another pass
    // over a slot's weights finds them in the caches (4-bit, 64 slots of 4096 x
    // 2048: 12 rows 97 us by one block, 116 by two; 30 rows 170 by two, 318 by
    // four).  16-bit weights, twice to four times the bytes, want one pass rather
    // (64 slots of 1536 x 1024, 12 rows: 44 and 40 us), and so do few workgroups,
    // where a pass is latency (one matrix of 4096 x 4096, 64 rows: 23 us by two
    // blocks, 20 by four; groups of 32 would spill).
    const int mb = mean <= (WT ? 16 : 8) || a.rows.R <= 16 ? 1 : !few || a.rows.R <= 32 || PER == 1 ? 2 : 4;
    const int segs = (a.K + kSegment - 1) / kSegment, turns = (segs + kStreamWaves - 1) / kStreamWaves;
    const int waves = (segs + turns - 1) / turns;
    // one tile a workgroup where two would leave CUs without one
    const int columns = act || few ? tiles : (tiles + 1) / 2;
    // Rows that a workgroup walks: one pass where a slot that holds most rows would
    // be walked longer than all workgroups take, 1280 of them at a time (128 slots of
    // 1408 x 1408, 1536 rows: 105 us in even slots both ways, 270 and 115 us with half
    // of them in one; one 4-bit matrix of 1536 x 2048, 16384 rows: 3.7 and 0.79 ms).
    // Else all of a slot's, as the other workgroups would only look for rows.
    const int blocks = (a.rows.R + 16 * mb - 1) / (16 * mb);
    StreamArgs t = a;
    t.slots = slots;
    t.unit_shift = mb == 1 ? 4 : mb == 2 ? 5 : 6;
    const int most = blocks > 3 && blocks > 1 + (long long)columns * slots / 1280 ? 32768 : 1;  // units of a slot
    while ((a.rows.R - 1) >> t.unit_shift >= most) ++t.unit_shift;
    const dim3 grid(columns, slots + ((a.rows.R - 1) >> t.unit_shift));
    if (act) return stream_launch_rows<WT, DT, 2, PER, true, EPI>(t, mb, grid, waves, s);
    if (few) return stream_launch_rows<WT, DT, 1, PER, false, EPI>(t, mb, grid, waves, s);
    return stream_launch_rows<WT, DT, 2, PER, false, EPI>(t, mb, grid, waves, s);
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

hipError_t launch_stream_bias_bf16(const StreamArgs& a, int act, hipStream_t s);
hipError_t launch_stream_bias_f16(const StreamArgs& a, int act, hipStream_t s);
hipError_t launch_stream_bf16(const StreamArgs& a, int w4, int act, hipStream_t s);
hipError_t launch_stream_f16(const StreamArgs& a, int w4, int act, hipStream_t s);

}  // namespace qmoe
