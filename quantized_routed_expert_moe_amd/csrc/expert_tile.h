// Expert products over whole tiles: the grouped matrix products of prompts
// and of training, forward (y = x w^T), data gradient (y = x w) and weight
// gradient (dw = dy^T x), as one tiled kernel.
//
// Bound by the matrix cores (2 R N K flops) once a slot has more than about a
// hundred rows, below that by the weights' stream.
//
// A workgroup computes a BQ x BP tile of the output; BP runs along the
// output's contiguous dimension.  v_mfma_f32_32x32x16 takes the P operand as
// its A matrix, so a lane ends with four consecutive output columns of one
// row and the epilogue packs them without shuffles.  The contraction advances
// 64 a stage through two LDS buffers, filled by global_load_lds_dwordx4 (no
// register staging) while the other is multiplied.
//
// Operands lie in LDS as they lie in memory:
//   direct      [row][64 of the contraction]: 128-byte rows; chunk (16 bytes) c
//               of row r at position c ^ (r % 8), so that ds_read_b128 of eight
//               rows at one c hits eight bank groups.
//   transposed  [64 of the contraction][row]: the contraction is the stored row
//               (w in the data gradient, both operands of the weight gradient);
//               ds_read_b64_tr_b16 hands a lane four contraction values of one
//               column.  Chunk c of row r at c ^ 4 (r % 4).
// Rows and columns outside the tile repeat its last one (their products are
// not stored); the contraction's rest is read from 16 zero bytes on both
// sides, so it adds nothing whatever the memory behind an operand holds.
//
// Row blocks of 32 past the tile's rows are neither loaded nor multiplied: the
// two wave rows own alternate blocks and the loop is instantiated for each
// count, so a ragged slot costs its rows rounded up to 64, not to the tile.
#pragma once
#include <type_traits>

#include "expert_ops.h"

namespace qmoe {

struct TileArgs {
    const void* q;    // rows of the output: x (forward, data gradient) or dy
    const void* p;    // columns of the output: w, or x in the weight gradient
    size_t p_stride;  // bytes from slot to slot (w)
    int N, K;         // of w
    RowMap rows;
    int q_rows, p_rows;  // row modes of q and (weight gradient) p
    int y_rows;
    void* y;
    int y_f32;
    int splits;       // weight gradient: parts of a slot's rows
};

enum { kForward = 0, kDataGrad = 1, kWeightGrad = 2 };

__device__ __attribute__((aligned(16))) const uint32_t kZeroChunk[4] = {0, 0, 0, 0};

template <int DT>
__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
    if constexpr (DT == MOE_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Four consecutive values in their output type, from fp32 (one rounding).
template <int DT>
__device__ __forceinline__ uint2 pack4(const float* v) {
    typedef typename DType<DT>::type E;
    typedef E e4 __attribute__((ext_vector_type(4)));
    e4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = (E)v[i];
    return __builtin_bit_cast(uint2, u);
}

// QI x PI blocks of 32 x 32 a wave, WQ x WP waves.
template <int DT, int MODE, bool SWI, int QI, int PI, int WQ, int WP>
struct Tile {
    static constexpr int W = WQ * WP, THREADS = 64 * W;
    static constexpr int BQ = 32 * QI * WQ, BP = 32 * PI * WP;
    static constexpr bool QT = MODE == kWeightGrad, PT = MODE != kForward;  // transposed operands
    static constexpr int UNITS = 4;  // 1 KB loads a wave issues for an operand's stage
    static_assert(BQ / 8 == UNITS * W && BP / 8 == UNITS * W, "a stage is four loads a wave for each operand");
    static constexpr int STAGE = BQ * 128;  // bytes of an operand's stage

    // Source rows and chunk of a transposed operand's loads by this lane.
    template <int B>
    static __device__ __forceinline__ int tr_row(int wave, int lane, int i) {
        return (512 / B) * (wave + W * i) + lane / (B / 8);
    }
    template <int B>
    static __device__ __forceinline__ int tr_chunk(int wave, int lane) {
        return (lane % (B / 8)) ^ (4 * (tr_row<B>(wave, lane, 0) & 3));
    }

    static __device__ __forceinline__ void dma(const uint8_t* src, uint8_t* lds) {
        __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
    }
};

template <int DT, int MODE, bool SWI, int QI, int PI, int WQ, int WP, int NB>
__device__ __forceinline__ void tile_product(const TileArgs& a, int slot, int q0, int nq, int c0, int p0, int len,
                                             uint8_t* sq0, uint8_t* sq1, uint8_t* sp0, uint8_t* sp1,
                                             f32x16 (&acc)[NB][PI]) {
    typedef Tile<DT, MODE, SWI, QI, PI, WQ, WP> C;
    constexpr int W = C::W, U = C::UNITS;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave % WQ, wp = wave / WQ;
    const int N = a.N, K = a.K;
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(kZeroChunk);
    // loads of the Q operand that hold rows of the blocks in use
    constexpr int UQ = C::QT ? U : (NB * 32 * WQ + 8 * W - 1) / (8 * W);

    // ---- addresses of the stage's loads.  Rows and columns outside the tile
    // repeat its last one: their products are never stored.
    const uint8_t* qp[U];  // direct: this lane's row and chunk at contraction 0
    const uint8_t* pp[U];
    int qr[U], pr[U];      // weight gradient: source rows of the next stage
    const int dchunk = (lane & 7) ^ (lane >> 3);
    const uint8_t* w = static_cast<const uint8_t*>(a.p) + (MODE == kWeightGrad ? 0 : (size_t)slot * a.p_stride);
    if constexpr (C::QT) {
        qp[0] = static_cast<const uint8_t*>(a.q) + (size_t)min(q0 + 8 * C::template tr_chunk<C::BQ>(wave, lane), N - 8) * 2;
    } else {
        const int ld = MODE == kForward ? K : N;
#pragma unroll
        for (int i = 0; i < UQ; ++i) {
            const int r = min(8 * (wave + W * i) + (lane >> 3), nq - 1);
            qp[i] = static_cast<const uint8_t*>(a.q) + ((size_t)row_of(a.rows, a.q_rows, q0 + r) * ld + 8 * dchunk) * 2;
        }
    }
    if constexpr (C::PT) {
        pp[0] = w + (size_t)min(p0 + 8 * C::template tr_chunk<C::BP>(wave, lane), K - 8) * 2;
        if (MODE == kDataGrad) pp[0] += (size_t)C::template tr_row<C::BP>(wave, lane, 0) * K * 2;
    } else {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int r = 8 * (wave + W * i) + (lane >> 3);
            int n = min(p0 + r, N - 1);
            // each wave's 64 columns: 32 gate rows, then the 32 up rows of the same features
            if (SWI) n = min(p0 + (r / 64) * 32 + r % 32, N / 2 - 1) + (r % 64 < 32 ? 0 : N / 2);
            pp[i] = w + ((size_t)n * K + 8 * dchunk) * 2;
        }
    }
    // source rows of the weight gradient's stage st
    auto fetch_rows = [&](int st) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            qr[i] = row_of(a.rows, a.q_rows, c0 + min(st * 64 + C::template tr_row<C::BQ>(wave, lane, i), len - 1));
            pr[i] = row_of(a.rows, a.p_rows, c0 + min(st * 64 + C::template tr_row<C::BP>(wave, lane, i), len - 1));
        }
    };
    const int stages = (len + 63) / 64;
    // REST: the last stage, cut by the contraction's end
    auto load_part = [&](int st, uint8_t* sq, uint8_t* sp, auto rest) {
        constexpr bool REST = decltype(rest)::value;
#pragma unroll
        for (int i = 0; i < UQ; ++i) {
            const uint8_t* src;
            bool in;
            if constexpr (C::QT) {
                src = qp[0] + (size_t)qr[i] * N * 2;
                in = st * 64 + C::template tr_row<C::BQ>(wave, lane, i) < len;
            } else {
                src = qp[i] + (size_t)st * 128;
                in = st * 64 + 8 * dchunk < len;
            }
            C::dma(!REST || in ? src : zero, sq + (wave + W * i) * 1024);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint8_t* src;
            bool in = st * 64 + C::template tr_row<C::BP>(wave, lane, i) < len;
            if constexpr (MODE == kWeightGrad) {
                src = pp[0] + (size_t)pr[i] * K * 2;
            } else if constexpr (C::PT) {
                src = pp[0] + (size_t)(st * 64 + (512 / C::BP) * W * i) * K * 2;
            } else {
                src = pp[i] + (size_t)st * 128;
                in = st * 64 + 8 * dchunk < len;
            }
            C::dma(!REST || in ? src : zero, sp + (wave + W * i) * 1024);
        }
    };
    auto load = [&](int st, uint8_t* sq, uint8_t* sp) {
        if (st * 64 + 64 <= len) load_part(st, sq, sp, std::false_type{});
        else load_part(st, sq, sp, std::true_type{});
    };

    // ---- fragment reads: k16 step s, block b of the wave
    const int swz = lane & 7, khalf = lane >> 5;
    const int trow = 8 * khalf + ((lane & 15) >> 2);  // first contraction row of a transposed read
    const int tcol = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    auto direct = [&](const uint8_t* s, int row, int step) {
        return *reinterpret_cast<const uint4*>(s + (row + (lane & 31)) * 128 + (((2 * step + khalf) ^ swz) * 16));
    };
    auto transposed = [&](const uint8_t* s, int col, int step, int width) {
        const int at = (16 * step + trow) * width * 2 + (((col / 8 + tcol) ^ (4 * (trow & 3))) * 16) + (lane & 1) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(s + at));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(s + at + 4 * width * 2));
        const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
        return make_uint4(l.x, l.y, h.x, h.y);
    };
    auto multiply = [&](const uint8_t* sq, const uint8_t* sp) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint4 fq[NB], fp[PI];
#pragma unroll
            for (int p = 0; p < PI; ++p) {
                const int col = 32 * (wp * PI + p);
                fp[p] = C::PT ? transposed(sp, col, s, C::BP) : direct(sp, col, s);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int row = 32 * (wq + WQ * b);
                fq[b] = C::QT ? transposed(sq, row, s, C::BQ) : direct(sq, row, s);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int p = 0; p < PI; ++p) acc[b][p] = mfma32<DT>(fp[p], fq[b], acc[b][p]);
        }
    };
    if (stages == 0) return;
    if (MODE == kWeightGrad) fetch_rows(0);
    load(0, sq0, sp0);
    if (MODE == kWeightGrad) fetch_rows(1);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();
    int st = 0;
    for (; st + 1 < stages; st += 2) {
        load(st + 1, sq1, sp1);
        if (MODE == kWeightGrad) fetch_rows(st + 2);
        multiply(sq0, sp0);
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        if (st + 2 < stages) {
            load(st + 2, sq0, sp0);
            if (MODE == kWeightGrad) fetch_rows(st + 3);
        }
        multiply(sq1, sp1);
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
    }
    if (st < stages) multiply(sq0, sp0);
}

// The tile's rows, rounded and stored.
template <int DT, int MODE, bool SWI, int QI, int PI, int WQ, int WP, int NB>
__device__ __forceinline__ void tile_store(const TileArgs& a, int slot, int q0, int nq, int p0, uint8_t* sq0, uint8_t* sq1,
                                           uint8_t* sp0, uint8_t* sp1, const f32x16 (&acc)[NB][PI]) {
    typedef Tile<DT, MODE, SWI, QI, PI, WQ, WP> C;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave % WQ, wp = wave / WQ, N = a.N, K = a.K;
    const int width = MODE == kForward ? (SWI ? N / 2 : N) : K;
    // Epilogue: a block of 32 rows at a time through the wave's share of the
    // stage buffers, out in 16-byte pieces of whole rows.
    __syncthreads();
    constexpr int WCOLS = SWI ? 32 * PI / 2 : 32 * PI;  // columns of the wave
    static_assert(!SWI || PI == 2, "gate and up blocks of the same features");
    constexpr int SHARE = 4 * C::STAGE / C::W;
    static_assert(SHARE >= 32 * (WCOLS * 4 + 16), "a block of fp32 rows fits the wave's share");
    const int buf = wave * 4 / C::W;
    uint8_t* mine = (buf == 0 ? sq0 : buf == 1 ? sq1 : buf == 2 ? sp0 : sp1) + (wave % (C::W / 4)) * SHARE;
    const int col0 = p0 + wp * WCOLS;
    const int es = a.y_f32 ? 4 : 2, stride = WCOLS * es + 16;
    const int lanes = WCOLS * es / 16, row_in = lane / lanes, piece = lane % lanes, rows_at = 64 / lanes;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int base = 32 * (wq + WQ * b);
        if (base >= nq) continue;
#pragma unroll
        for (int p = 0; p < (SWI ? 1 : PI); ++p)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = acc[b][p][4 * g + e];
                    if (SWI) v[e] = v[e] * sigmoid_f32(v[e]) * acc[b][PI - 1][4 * g + e];
                }
                const int c = 32 * p + 8 * g + 4 * (lane >> 5);
                uint8_t* at = mine + (lane & 31) * stride + c * es;
                if (a.y_f32) *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
                else *reinterpret_cast<uint2*>(at) = pack4<DT>(v);
            }
        for (int r0 = 0; r0 < 32; r0 += rows_at) {
            const int r = r0 + row_in, row = base + r, c = col0 + piece * (16 / es);
            const uint4 v = *reinterpret_cast<const uint4*>(mine + r * stride + piece * 16);
            if (row >= nq || c >= width) continue;
            const size_t out = MODE == kWeightGrad ? ((size_t)slot * N + q0 + row) * K + c
                                                   : (size_t)row_of(a.rows, a.y_rows, q0 + row) * width + c;
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.y) + out * es) = v;
        }
    }
}

// Row tile `index` of the batch: whole tiles of every slot first, then the
// slots' rests.  Found by one scan over the slots (S <= 1024) in LDS.
template <int BQ, int THREADS>
__device__ __forceinline__ bool find_tile(const RowMap& m, int index, int& slot, int& q0, int& nq) {
    __shared__ int wsum[2][THREADS / 64], found[3];
    constexpr int PER = 1024 / THREADS;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int2 r[PER];
    int whole = 0, rest = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int s = t * PER + j;
        r[j] = s < m.S ? slot_range(m, s) : make_int2(0, 0);
        whole += r[j].y / BQ;
        rest += r[j].y % BQ != 0;
    }
    int iw = whole, ir = rest;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(iw, o, 64), y = __shfl_up(ir, o, 64);
        if (lane >= o) {
            iw += x;
            ir += y;
        }
    }
    if (lane == 63) {
        wsum[0][wave] = iw;
        wsum[1][wave] = ir;
    }
    if (t == 0) found[0] = -1;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) {
            iw += wsum[0][w];
            ir += wsum[1][w];
        }
        total += wsum[0][w];
    }
    iw -= whole;
    ir = ir - rest + total;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int n = r[j].y / BQ, left = r[j].y % BQ;
        if (index >= iw && index < iw + n) {
            found[0] = t * PER + j;
            found[1] = r[j].x + (index - iw) * BQ;
            found[2] = BQ;
        }
        iw += n;
        if (left) {
            if (index == ir) {
                found[0] = t * PER + j;
                found[1] = r[j].x + n * BQ;
                found[2] = left;
            }
            ++ir;
        }
    }
    __syncthreads();
    slot = __builtin_amdgcn_readfirstlane(found[0]);
    q0 = __builtin_amdgcn_readfirstlane(found[1]);
    nq = __builtin_amdgcn_readfirstlane(found[2]);
    return slot >= 0;
}

template <int DT, int MODE, bool SWI, int QI, int PI, int WQ, int WP>
__global__ __launch_bounds__(64 * WQ * WP) void expert_tile_kernel(const TileArgs a) {
    typedef Tile<DT, MODE, SWI, QI, PI, WQ, WP> C;
    // Four arrays, so that the compiler can tell the loads into one buffer
    // from the reads of the other.
    __shared__ __attribute__((aligned(16))) uint8_t sq0[C::STAGE], sq1[C::STAGE], sp0[C::STAGE], sp1[C::STAGE];
    const int N = a.N, K = a.K;
    // The column tiles of a row tile run on one XCD (workgroup number modulo
    // 8), which then serves the shared rows from its L2.
    const int width = MODE == kForward ? (SWI ? N / 2 : N) : K;  // columns of the output
    constexpr int COLS = SWI ? C::BP / 2 : C::BP;                // of them in a tile
    const int ptiles = (width + COLS - 1) / COLS;
    const int xcd = blockIdx.x & 7, j = blockIdx.x >> 3;
    const int p0 = (j % ptiles) * COLS, qt = (j / ptiles) * 8 + xcd;
    int slot, q0, nq, c0 = 0, len;
    if (MODE == kWeightGrad) {
        const int ntiles = (N + C::BQ - 1) / C::BQ;
        const int part = qt / (ntiles * a.rows.S), st = qt % (ntiles * a.rows.S);
        if (part >= a.splits) return;
        slot = st / ntiles;
        q0 = (st % ntiles) * C::BQ;
        nq = min(C::BQ, N - q0);
        const int2 r = slot_range(a.rows, slot);
        const int per = ((r.y + a.splits - 1) / a.splits + 63) / 64 * 64;
        c0 = r.x + min(part * per, r.y);
        len = min(per, r.x + r.y - c0);
        slot += part * a.rows.S;
    } else {
        if (!find_tile<C::BQ, C::THREADS>(a.rows, qt, slot, q0, nq)) return;
        len = MODE == kForward ? K : N;
    }
    const int nb = (nq + 32 * WQ - 1) / (32 * WQ);
    auto body = [&](auto tag) {
        constexpr int NB = decltype(tag)::value;
        f32x16 acc[NB][PI] = {};
        tile_product<DT, MODE, SWI, QI, PI, WQ, WP, NB>(a, slot, q0, nq, c0, p0, len, sq0, sq1, sp0, sp1, acc);
        tile_store<DT, MODE, SWI, QI, PI, WQ, WP, NB>(a, slot, q0, nq, p0, sq0, sq1, sp0, sp1, acc);
    };
    if (MODE == kWeightGrad || nb == QI) body(std::integral_constant<int, QI>{});
    else if (nb == 1) body(std::integral_constant<int, 1>{});
    else if (QI > 2 && nb == 2) body(std::integral_constant<int, QI < 2 ? QI : 2>{});
    else if (QI > 3 && nb == 3) body(std::integral_constant<int, QI < 3 ? QI : 3>{});
}

template <int DT, int MODE, bool SWI, int QI, int PI, int WQ, int WP>
static hipError_t tile_launch(const TileArgs& a, hipStream_t s) {
    typedef Tile<DT, MODE, SWI, QI, PI, WQ, WP> C;
    const int width = MODE == kForward ? (SWI ? a.N / 2 : a.N) : a.K;
    constexpr int COLS = SWI ? C::BP / 2 : C::BP;
    const long long ptiles = (width + COLS - 1) / COLS;
    const long long qtiles = MODE == kWeightGrad
                                 ? (long long)((a.N + C::BQ - 1) / C::BQ) * a.rows.S * a.splits
                                 : a.rows.R / C::BQ + (a.rows.R < a.rows.S ? a.rows.R : a.rows.S);
    const long long grid = (qtiles + 7) / 8 * 8 * ptiles;
    if (grid > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    expert_tile_kernel<DT, MODE, SWI, QI, PI, WQ, WP><<<dim3((uint32_t)grid), C::THREADS, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
static hipError_t tile_launch_type(const TileArgs& a, int mode, int act, int big, hipStream_t s) {
    if (mode == kForward && act) return big ? tile_launch<DT, kForward, true, 4, 2, 2, 4>(a, s) : tile_launch<DT, kForward, true, 2, 2, 2, 2>(a, s);
    if (mode == kForward) return big ? tile_launch<DT, kForward, false, 4, 2, 2, 4>(a, s) : tile_launch<DT, kForward, false, 2, 2, 2, 2>(a, s);
    if (mode == kDataGrad) return big ? tile_launch<DT, kDataGrad, false, 4, 2, 2, 4>(a, s) : tile_launch<DT, kDataGrad, false, 2, 2, 2, 2>(a, s);
    return big ? tile_launch<DT, kWeightGrad, false, 4, 2, 2, 4>(a, s) : tile_launch<DT, kWeightGrad, false, 2, 2, 2, 2>(a, s);
}

hipError_t launch_tile_bf16(const TileArgs& a, int mode, int act, int big, hipStream_t s);
hipError_t launch_tile_f16(const TileArgs& a, int mode, int act, int big, hipStream_t s);

}  // namespace qmoe
