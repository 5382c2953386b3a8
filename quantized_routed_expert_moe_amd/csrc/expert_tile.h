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
// row and the epilogue packs them without shuffles.  256 x 256 by eight waves of
// 128 x 64 where such tiles fill the chip, else 128 x 128 by four of 64 x 64.
// Measured for 8192 x 8192 x 8192 (bf16): 1340 TFLOP/s forward, 1350 data
// gradient, 1300 weight gradient; four waves of 128 x 128, rings of more and
// shorter stages and two 256 x 128 tiles a CU were slower.
//
// The contraction advances 64 a stage through two LDS buffers, filled by
// global_load_lds_dwordx4 (no register staging).  A stage is four steps of 16;
// the fragments of the next step are read while this step multiplies, the last
// step's already from the other buffer: the one barrier of a stage stands
// before it, and behind the barrier the buffer just read is filled again.
//
// Operands lie in LDS as they lie in memory:
//   direct      [row][64 of the contraction]: 128-byte rows; chunk (16 bytes) c
//               of row r at position c ^ (r / 2) % 8: LDS has 64 banks of 4
//               bytes and ds_read_b128 takes 16 lanes at a time, whose 16 rows at
//               one c then cover the 256 bytes once (c ^ r % 8 measured half of
//               all LDS cycles as conflicts).
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

#include "act.h"
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
    int group;        // column tiles of a group
    Epilogue epi;     // biased products
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
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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

// QI x PI blocks of 32 x 32 a wave, WQ x WP waves.  EPI: the store adds bias and residual.
template <int DT_, int MODE_, bool SWI_, int QI_, int PI_, int WQ_, int WP_, bool EPI_ = false>
struct Tile {
    static constexpr int DT = DT_, MODE = MODE_, QI = QI_, PI = PI_, WQ = WQ_, WP = WP_, NBUF = 2;
    static constexpr bool SWI = SWI_, EPI = EPI_;
    static constexpr int BK = 64;
    static constexpr int W = WQ * WP, THREADS = 64 * W;
    static constexpr int BQ = 32 * QI * WQ, BP = 32 * PI * WP;
    static constexpr bool QT = MODE == kWeightGrad, PT = MODE != kForward;  // transposed operands
    static constexpr int UQ = BQ / 8 / W, UP = BP / 8 / W;  // 1 KB loads of a wave for a stage
    static constexpr int QBYTES = BQ * 2 * BK, PBYTES = BP * 2 * BK;
    static constexpr int COLS = SWI ? BP / 2 : BP;  // output columns of a tile
    static constexpr int WINDOW = 1024;             // weight gradient: source rows held in LDS
    static_assert(W % 2 == 0, "a load's rows keep their place in the swizzle");
    static_assert(!SWI || PI % 2 == 0, "gate and up blocks of the same features");
    static_assert(UQ * W * 8 == BQ && UP * W * 8 == BP, "whole loads");
};

// Transposed operand of B columns: row of the stage and chunk that this lane
// of load i brings.
template <int B, int W>
__device__ __forceinline__ int tr_row(int wave, int lane, int i) {
    return (512 / B) * (wave + W * i) + lane / (B / 8);
}
template <int B, int W>
__device__ __forceinline__ int tr_chunk(int wave, int lane) {
    return (lane % (B / 8)) ^ (4 * (tr_row<B, W>(wave, lane, 0) & 3));
}

__device__ __forceinline__ void load_to_lds(const uint8_t* src, uint8_t* lds) {
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// s_waitcnt vmcnt(N), other counters unconstrained.
template <int N>
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// Every wave's LDS traffic before it is done, none after it has begun; loads
// to LDS in flight are not waited for.
__device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// LOADS loads to LDS spread evenly behind M matrix instructions, READS LDS
// reads behind the first half of them: their values are due next.
template <int M, int READS, int LOADS, int I = 0>
__device__ __forceinline__ void spread() {
    if constexpr (I < M) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        constexpr int H = (M + 1) / 2, reads = I < H ? READS * (I + 1) / H - READS * I / H : 0;
        constexpr int loads = LOADS * (I + 1) / M - LOADS * I / M;
        if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
        if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x010, loads, 0);
        spread<M, READS, LOADS, I + 1>();
    }
}

// Fragment of a transposed operand of `width` columns: step of 16 of the
// contraction, block of 32 columns from `col` on.
__device__ __forceinline__ uint4 read_transposed(const uint8_t* s, int lane, int col, int step, int width) {
    const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);  // first contraction row of the read
    const int chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int at = (16 * step + row) * width * 2 + (((col / 8 + chunk) ^ (4 * (row & 3))) * 16) + (lane & 1) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(s + at));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(s + at + 4 * width * 2));
    const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
    return make_uint4(l.x, l.y, h.x, h.y);
}

template <typename C>
struct TileLds {
    uint8_t* q[C::NBUF];
    uint8_t* p[C::NBUF];
    int32_t* row[2];  // weight gradient: source rows of dy and x for the window
};

template <typename C, int NB>
__device__ __forceinline__ void tile_product(const TileArgs& a, int slot, int q0, int nq, int c0, int p0, int len,
                                             const TileLds<C>& lds, f32x16 (&acc)[NB][C::PI]) {
    constexpr int W = C::W, WQ = C::WQ, PI = C::PI, MODE = C::MODE, BK = C::BK;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave % WQ, wp = wave / WQ;
    const int N = a.N, K = a.K;
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(kZeroChunk);
    // loads of the Q operand that hold rows of the blocks in use
    constexpr int UQ = C::QT ? C::UQ : (NB * 32 * WQ + 8 * W - 1) / (8 * W), UP = C::UP;

    // This lane's part of every address: a 64-bit address of a row of x or dy
    // (they may pass 4 GB), a 32-bit offset into a slot's matrix (at most 2 GB).
    // What advances with the stage is added to the uniform part.
    const uint8_t* qp[C::UQ];  // direct: row and chunk at contraction 0; transposed: column
    uint32_t po[C::UP];
    const int dchunk = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));  // (r / 2) % 8 of its row r = 8 (wave + W i) + lane / 8
    const uint8_t* w = static_cast<const uint8_t*>(a.p) + (MODE == kWeightGrad ? 0 : (size_t)slot * a.p_stride);
    if constexpr (C::QT) {
        qp[0] = static_cast<const uint8_t*>(a.q) + (size_t)min(q0 + 8 * tr_chunk<C::BQ, W>(wave, lane), N - 8) * 2;
    } else {
        const int ld = MODE == kForward ? K : N;
#pragma unroll
        for (int i = 0; i < UQ; ++i) {
            const int r = min(8 * (wave + W * i) + (lane >> 3), nq - 1);
            qp[i] = static_cast<const uint8_t*>(a.q) + ((size_t)row_of(a.rows, a.q_rows, q0 + r) * ld + 8 * dchunk) * 2;
        }
    }
    if constexpr (C::PT) {
        po[0] = (uint32_t)min(p0 + 8 * tr_chunk<C::BP, W>(wave, lane), K - 8) * 2;
        if (MODE == kDataGrad) po[0] += (uint32_t)tr_row<C::BP, W>(wave, lane, 0) * (uint32_t)K * 2;
    } else {
#pragma unroll
        for (int i = 0; i < UP; ++i) {
            const int r = 8 * (wave + W * i) + (lane >> 3);
            int n = min(p0 + r, N - 1);
            // of each 64 columns 32 gate rows, then the 32 up rows of the same features
            if (C::SWI) n = min(p0 + (r / 64) * 32 + r % 32, N / 2 - 1) + (r % 64 < 32 ? 0 : N / 2);
            po[i] = ((uint32_t)n * (uint32_t)K + 8 * dchunk) * 2;
        }
    }
    const int stages = max((len + BK - 1) / BK, 4);  // the last three may hold zeros only
    // weight gradient: source rows of dy and x, a ring that is filled half a
    // window at a time well ahead of the loads
    int filled = 0;
    auto fill_rows = [&](int n) {
        for (int i = threadIdx.x; i < n; i += C::THREADS) {
            const int q = c0 + min(filled + i, len - 1), at = (filled + i) % C::WINDOW;
            lds.row[0][at] = row_of(a.rows, a.q_rows, q);
            lds.row[1][at] = row_of(a.rows, a.p_rows, q);
        }
        filled += n;
        __syncthreads();
    };
    auto refill = [&](int st) {  // before the loads of stages st + 2 and st + 3
        if (MODE == kWeightGrad && filled < len && (st + 4) * BK > filled) fill_rows(C::WINDOW / 2);
    };
    // Slots begin the contraction at different stages: at one stage all CUs
    // would read the same 128 bytes of their rows, and rows of 2^n bytes put
    // those into a few memory channels (128 slots of 64 rows, 1536 x 2048: 206 us
    // in step, 159 us so; the data gradient reads whole rows, 163 and 165 us).
    // The order of a row's sums then depends on its slot's number alone.
    const int wholes = len / BK;
    const int rotation = MODE == kForward && wholes > 0 ? (int)(5u * (uint32_t)slot % (uint32_t)wholes) : 0;
    // Stage st's loads.  No branch, so that they can stand between matrix
    // instructions.  REST: what lies behind the contraction's end is selected
    // away (the stage may lie behind it as a whole); else the stage is whole.
    auto load = [&](int st, int buf, auto rest) {
        constexpr bool REST = decltype(rest)::value;
        uint8_t *sq = lds.q[buf], *sp = lds.p[buf];
        if (MODE == kForward && st < wholes) st = st + rotation < wholes ? st + rotation : st + rotation - wholes;
        uint32_t k0 = (uint32_t)st * BK;
        asm("" : "+s"(k0));  // keeps the addresses out of the loop's registers
        const int left = len - (int)k0;
#pragma unroll
        for (int i = 0; i < UQ; ++i) {
            const uint8_t* src;
            bool in;
            if constexpr (C::QT) {
                const int r = tr_row<C::BQ, W>(wave, lane, i);
                src = qp[0] + (size_t)(uint32_t)lds.row[0][(k0 + r) % C::WINDOW] * (uint32_t)(N * 2);
                in = r < left;
            } else {
                src = qp[i] + (size_t)k0 * 2;
                in = 8 * dchunk < left;
            }
            load_to_lds(!REST || in ? src : zero, sq + (wave + W * i) * 1024);
        }
#pragma unroll
        for (int i = 0; i < UP; ++i) {
            const uint8_t* src;
            const int r = tr_row<C::BP, W>(wave, lane, i);
            bool in = r < left;
            if constexpr (MODE == kWeightGrad) {
                src = w + po[0] + (size_t)(uint32_t)lds.row[1][(k0 + r) % C::WINDOW] * (uint32_t)(K * 2);
            } else if constexpr (C::PT) {
                src = w + (size_t)(k0 + (512 / C::BP) * W * i) * (uint32_t)(K * 2) + po[0];
            } else {
                src = w + (size_t)k0 * 2 + po[i];
                in = 8 * dchunk < left;
            }
            load_to_lds(!REST || in ? src : zero, sp + (wave + W * i) * 1024);
        }
    };

    // ---- fragment reads: step of 16, block of 32 rows or columns
    const int khalf = lane >> 5, swz = (lane >> 1) & 7;
    auto direct = [&](const uint8_t* s, int row, int step) {
        return *reinterpret_cast<const uint4*>(s + (row + (lane & 31)) * 128 + (((2 * step + khalf) ^ swz) * 16));
    };
    uint4 fq[2][NB], fp[2][PI];
    auto read = [&](int set, int buf, int step) {
#pragma unroll
        for (int p = 0; p < PI; ++p) {
            const int col = 32 * (wp * PI + p);
            fp[set][p] = C::PT ? read_transposed(lds.p[buf], lane, col, step, C::BP) : direct(lds.p[buf], col, step);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int row = 32 * (wq + WQ * b);
            fq[set][b] = C::QT ? read_transposed(lds.q[buf], lane, row, step, C::BQ) : direct(lds.q[buf], row, step);
        }
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int p = 0; p < PI; ++p) acc[b][p] = mfma32<C::DT>(fp[set][p], fq[set][b], acc[b][p]);
    };
    constexpr int READS = (C::PT ? 2 : 1) * PI + (C::QT ? 2 : 1) * NB;
    if (MODE == kWeightGrad) fill_rows(min(C::WINDOW, stages * BK));
    enum { kWhole, kRest, kNext, kLast };
    // Steps 0 to 3 of a stage.  kWhole, kRest: stage st + 2 exists, its loads
    // stand between the last step's matrix instructions.  kLast: nothing follows.
    auto stage = [&](int st, int buf, auto kind) {
        constexpr int KIND = decltype(kind)::value;
        constexpr bool LOADS = KIND == kWhole || KIND == kRest;
#pragma unroll
        for (int step = 0; step < 3; ++step) {
            read((step + 1) & 1, buf, step + 1);
            multiply(step & 1);
            spread<NB * PI, READS, 0>();
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (KIND != kLast) {
            __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0): the other buffer is whole, this one is read
            stage_barrier();
            if constexpr (LOADS) load(st + 2, buf, std::integral_constant<bool, KIND == kRest>{});
            read(0, buf ^ 1, 0);
            multiply(1);
            spread<NB * PI, READS, LOADS ? UQ + UP : 0>();
        } else {
            multiply(1);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // An odd count puts its first stage, alone, into buffer 1; pairs follow, the
    // last two apart (the second of them brings the contraction's rest).  A test
    // of the count behind the loop would leave two copies of the accumulators.
    auto begin = [&](int buf) {
        load(0, buf, std::true_type{});
        __builtin_amdgcn_sched_barrier(0);
        load(1, buf ^ 1, std::true_type{});
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<UQ + UP>();  // stage 0's
        stage_barrier();
        read(0, buf, 0);
    };
    const std::integral_constant<int, kWhole> whole;
    const std::integral_constant<int, kRest> cut;
    int st = stages & 1;
    if (st) {
        begin(1);
        stage(0, 1, cut);
    } else {
        begin(0);
    }
    for (; st + 4 < stages; st += 2) {
        refill(st);
        stage(st, 0, whole);
        stage(st + 1, 1, whole);
    }
    refill(st);
    stage(st, 0, cut);
    stage(st + 1, 1, cut);
    stage(st + 2, 0, std::integral_constant<int, kNext>{});
    stage(st + 3, 1, std::integral_constant<int, kLast>{});
}

// A weight gradient tile of a slot with at most 64 rows: one stage, and of it
// only the steps of 16 rows that exist; a lane loads its row numbers itself.
template <typename C>
__device__ __forceinline__ void tile_short(const TileArgs& a, int q0, int c0, int p0, int len, const TileLds<C>& lds,
                                           f32x16 (&acc)[C::QI][C::PI]) {
    constexpr int W = C::W;
    static_assert(16 * C::UQ == C::BK && 16 * C::UP == C::BK, "a load of every wave brings a step");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave % C::WQ, wp = wave / C::WQ, steps = (len + 15) / 16;
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(kZeroChunk);
    const uint8_t* q = static_cast<const uint8_t*>(a.q) + (size_t)min(q0 + 8 * tr_chunk<C::BQ, W>(wave, lane), a.N - 8) * 2;
    const uint8_t* p = static_cast<const uint8_t*>(a.p) + (size_t)min(p0 + 8 * tr_chunk<C::BP, W>(wave, lane), a.K - 8) * 2;
#pragma unroll
    for (int i = 0; i < C::UQ; ++i) {
        if (i >= steps) continue;
        const int rq = tr_row<C::BQ, W>(wave, lane, i), rp = tr_row<C::BP, W>(wave, lane, i);
        const size_t from = (size_t)(uint32_t)row_of(a.rows, a.q_rows, c0 + min(rq, len - 1)) * (uint32_t)(a.N * 2);
        load_to_lds(rq < len ? q + from : zero, lds.q[0] + (wave + W * i) * 1024);
        const size_t with = (size_t)(uint32_t)row_of(a.rows, a.p_rows, c0 + min(rp, len - 1)) * (uint32_t)(a.K * 2);
        load_to_lds(rp < len ? p + with : zero, lds.p[0] + (wave + W * i) * 1024);
    }
    wait_loads<0>();
    __syncthreads();
#pragma unroll
    for (int step = 0; step < C::BK / 16; ++step) {
        if (step >= steps) continue;
        uint4 fq[C::QI], fp[C::PI];
#pragma unroll
        for (int b = 0; b < C::QI; ++b) fq[b] = read_transposed(lds.q[0], lane, 32 * (wq + C::WQ * b), step, C::BQ);
#pragma unroll
        for (int p = 0; p < C::PI; ++p) fp[p] = read_transposed(lds.p[0], lane, 32 * (wp * C::PI + p), step, C::BP);
#pragma unroll
        for (int b = 0; b < C::QI; ++b)
#pragma unroll
            for (int p = 0; p < C::PI; ++p) acc[b][p] = mfma32<C::DT>(fp[p], fq[b], acc[b][p]);
    }
}

// Weight gradient of a slot (or part) without rows: tile `tile` of `tiles` writes
// its share of the matrix's zeros.  A gradient that the last-level cache holds
// goes through it, a workgroup's runs of 16 bytes a thread in turn; a larger one
// past it, each wave in one run.  Slots without any row, us through and past: 45 of
// 1000 x 1400, fp32 (252 MB) 32 and 43; 12 of 2816 x 2048 (277 MB) 35 and 44, 45 (1.04
// GB) 169 and 158; 128 of 1408 x 2048 with 64 rows in all (1.5 GB) 253 and 225.  By the
// tiles' own rows odd widths cost twice as much (128 of 2064 x 472, bf16: 87 us, 39
// in runs).
template <typename C>
__device__ __forceinline__ void tile_zero(const TileArgs& a, int slot, int tile, int tiles) {
    const size_t units = (size_t)a.N * a.K / (a.y_f32 ? 4 : 8);  // of 16 bytes
    const size_t share = ((units + tiles - 1) / tiles + 63) & ~(size_t)63;
    const size_t from = min(units, tile * share), end = min(units, from + share);
    u32x4* y = static_cast<u32x4*>(a.y) + slot * units;
    const u32x4 zero = {0, 0, 0, 0};
    if (a.splits > 1 || a.rows.S * units <= (300u << 20) / 16) {
        for (size_t i = from + threadIdx.x; i < end; i += C::THREADS) y[i] = zero;
    } else {
        const size_t run = (end - from) / (C::W * 64) * 64;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const size_t to = wave == C::W - 1 ? end : from + (wave + 1) * run;
        for (size_t i = from + wave * run + lane; i < to; i += 64) __builtin_nontemporal_store(zero, y + i);
    }
}

// The tile's rows, rounded and stored: a block of 32 rows at a time through
// the wave's share of the stage buffers, out in 16-byte pieces of whole rows.
template <typename C, int NB>
__device__ __forceinline__ void tile_store(const TileArgs& a, int slot, int q0, int nq, int p0, const TileLds<C>& lds,
                                           const f32x16 (&acc)[NB][C::PI]) {
    constexpr int PI = C::PI, WQ = C::WQ, SHARE = 32 * (128 + 16), PERQ = C::QBYTES / SHARE, PERP = C::PBYTES / SHARE;
    static_assert(C::W <= PERQ * C::NBUF + PERP * C::NBUF, "a share for each wave");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave % WQ, wp = wave / WQ, N = a.N, K = a.K;
    const int width = C::MODE == kForward ? (C::SWI ? N / 2 : N) : K;
    uint8_t* mine = nullptr;
#pragma unroll
    for (int u = 0; u < C::NBUF; ++u) {
        if (wave >= u * PERQ && wave < (u + 1) * PERQ) mine = lds.q[u] + (wave - u * PERQ) * SHARE;
        const int v = wave - C::NBUF * PERQ;
        if (v >= u * PERP && v < (u + 1) * PERP) mine = lds.p[u] + (v - u * PERP) * SHARE;
    }
    __syncthreads();
    // PAST: stored past the caches.  Known to the compiler: of a store with and one
    // without the hint behind a branch it makes one without.
    auto block = [&](auto f32_tag, auto past_tag, int base, const f32x16 (&v)[PI], int p) {
        constexpr bool F32 = decltype(f32_tag)::value, PAST = decltype(past_tag)::value;
        constexpr int ES = F32 ? 4 : 2;
        // 128 bytes of a row: 32 fp32 columns, or the wave's 64 of a 16-bit type (SwiGLU leaves it 32)
        constexpr int BLOCKS = F32 || C::SWI ? 1 : 2, WIDE = 32 * BLOCKS, STRIDE = WIDE * ES + 16;
        constexpr int LANES = WIDE * ES / 16, AT = 64 / LANES;
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = v[p + j][4 * g + e];
                    if (C::SWI) o[e] = o[e] * sigmoid_f32(o[e]) * v[p + 1][4 * g + e];
                }
                uint8_t* at = mine + (lane & 31) * STRIDE + (32 * j + 8 * g + 4 * (lane >> 5)) * ES;
                if (F32) *reinterpret_cast<float4*>(at) = make_float4(o[0], o[1], o[2], o[3]);
                else *reinterpret_cast<uint2*>(at) = pack4<C::DT>(o);
            }
        const int piece = lane % LANES, c = p0 + wp * (C::SWI ? 16 * PI : 32 * PI) + (C::SWI ? 16 : 32) * p + piece * (16 / ES);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += AT) {
            const int r = r0 + lane / LANES, row = base + r;
            const uint4 u = *reinterpret_cast<const uint4*>(mine + r * STRIDE + piece * 16);
            if (row >= nq || c >= width) continue;
            const size_t out = C::MODE == kWeightGrad ? ((size_t)slot * N + q0 + row) * K + c
                                                      : (size_t)row_of(a.rows, a.y_rows, q0 + row) * width + c;
            uint8_t* at = static_cast<uint8_t*>(a.y) + out * ES;
            if constexpr (PAST)
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, u), reinterpret_cast<u32x4*>(at));
            else
                *reinterpret_cast<uint4*>(at) = u;
        }
    };
    auto rows = [&](auto f32_tag, auto past_tag) {
        constexpr int STEP = decltype(f32_tag)::value && !C::SWI ? 1 : 2;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int base = 32 * (wq + WQ * b);
            if (base >= nq) continue;
#pragma unroll
            for (int p = 0; p < PI; p += STEP) block(f32_tag, past_tag, base, acc[b], p);
        }
    };
    // A weight gradient is not read again soon: past the caches it takes 287
    // instead of 358 us (64 experts of 1536 x 2048, fp32, 280 to 2244 rows each).
    // Small tiles go through the caches where a row ends inside a line of 128
    // bytes, which would be written in two pieces (60 of 1072 x 1448, fp32, 27
    // rows each: 158 us past, 100 through; 128 of 1408 x 2048, 4 rows each: 221 us
    // past, 253 through), and with the parts that the next launch joins (256 x 256,
    // 32768 rows: 35.4 us past, 32.3 through).
    const std::true_type yes;
    const std::false_type no;
    if constexpr (C::MODE == kWeightGrad && C::BQ == 128) {
        const bool past = a.splits == 1 && K * (a.y_f32 ? 4 : 2) % 128 == 0;
        if (!a.y_f32) past ? rows(no, yes) : rows(no, no);
        else past ? rows(yes, yes) : rows(yes, no);
    } else {
        const std::bool_constant<C::MODE == kWeightGrad> past;
        a.y_f32 ? rows(yes, past) : rows(no, past);
    }
}

// LDS accesses of a wave's lanes before it come before those behind it: the hardware
// takes a wave's in order, the compiler is kept from moving them.
__device__ __forceinline__ void wave_lds_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// Eight elements of a row: fp32 or the tile's type.
template <int DT>
__device__ __forceinline__ void load8_of(const void* p, int f32, size_t at, float* v) {
    if (f32) load_vec8<MOE_F32>(p, at, v);
    else load_vec8<DT>(p, at, v);
}

// tile_store of a biased product.  32 rows of the wave's 64 columns at a time lie in its
// share of the stage buffers as fp32; a lane takes eight columns of a row, whose bias it holds
// in registers.  First z and the activation, in place, in a loop that is not unrolled (erf and
// the rest would be repeated 40 times in the code); then residual, rounding and store, the
// residual's rows requested before the first part.  With and without operands, us:
// 32768 pairs of 1536 x 2048 with SwiGLU 253 (bias, z) and 253, by tile_store 274; 2999 rows of
// 2048 x 4096 64 (bias, residual) and 62, by tile_store 60, with GELU 68.
template <typename C, int NB>
__device__ __forceinline__ void tile_store_epilogue(const TileArgs& a, int slot, int q0, int nq, int p0,
                                                    const TileLds<C>& lds, const f32x16 (&acc)[NB][C::PI]) {
    static_assert(C::MODE == kForward && C::PI == 2, "64 columns a wave");
    constexpr int DT = C::DT, WQ = C::WQ, STRIDE = 64 + 4, SHARE = 32 * STRIDE * 4;
    constexpr int PER = C::QBYTES / SHARE, LANES = C::SWI ? 4 : 8, AT = 64 / LANES, STEPS = 32 / AT;
    static_assert(C::QBYTES == C::PBYTES && C::W <= PER * 2 * C::NBUF, "a share for each wave");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave % WQ, wp = wave / WQ, N = a.N, width = C::SWI ? N / 2 : N;
    uint8_t* buf[4] = {lds.q[0], lds.q[1], lds.p[0], lds.p[1]};
    float* mine = nullptr;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (wave >= u * PER && wave < (u + 1) * PER) mine = reinterpret_cast<float*>(buf[u] + (wave - u * PER) * SHARE);
    const Epilogue& e = a.epi;
    const int piece = lane % LANES, c = p0 + wp * (C::SWI ? 32 : 64) + piece * 8;
    const bool in = c < width, early = C::SWI || e.act != MOE_ACT_NONE || e.z;
    float bias[C::SWI ? 16 : 8] = {};
    if (e.bias && in) {
        load8_of<DT>(e.bias, e.bias_f32, (size_t)slot * N + c, bias);
        if constexpr (C::SWI) load8_of<DT>(e.bias, e.bias_f32, (size_t)slot * N + width + c, bias + 8);
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int base = 32 * (wq + WQ * b);
        if (base >= nq) continue;
        size_t row[STEPS];
        bool live[STEPS];
        float res[STEPS][8];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int r = base + i * AT + lane / LANES;
            live[i] = in && r < nq;
            row[i] = (size_t)row_of(a.rows, a.y_rows, q0 + min(r, nq - 1));
            if (e.residual && live[i]) load8_of<DT>(e.residual, e.res_f32, row[i] * width + c, res[i]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x16 v = acc[b][j];
                *reinterpret_cast<float4*>(mine + (lane & 31) * STRIDE + 32 * j + 8 * g + 4 * (lane >> 5)) =
                    make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
            }
        wave_lds_order();
        if (early) {
#pragma unroll 1
            for (int i = 0; i < STEPS; ++i) {
                const int r = i * AT + lane / LANES;
                float* at = mine + r * STRIDE + piece * 8;
                float v[8];
                load_vec8<MOE_F32>(at, 0, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += bias[j];
                const bool store = e.z && in && base + r < nq;
                size_t out = 0;
                if (store) {
                    out = (size_t)row_of(a.rows, a.y_rows, q0 + base + r) * N + c;
                    store_vec8<DT>(e.z, out, v);
                }
                if constexpr (C::SWI) {
                    float u[8];
                    load_vec8<MOE_F32>(at + 32, 0, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] += bias[8 + j];
                    if (store) store_vec8<DT>(e.z, out + width, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] * sigmoid_f32(v[j]) * u[j];
                } else {
                    act8(e.act, v);
                }
                store_vec8<MOE_F32>(at, 0, v);
            }
            wave_lds_order();
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            float v[8];
            load_vec8<MOE_F32>(mine + (i * AT + lane / LANES) * STRIDE + piece * 8, 0, v);
            if (!live[i]) continue;
            if (!early) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += bias[j];
            }
            if (e.residual) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += res[i][j];
            }
            if (a.y_f32) store_vec8<MOE_F32>(a.y, row[i] * width + c, v);
            else store_vec8<DT>(a.y, row[i] * width + c, v);
        }
        wave_lds_order();
    }
}

// Row tile `index` of the batch, slots in order: whole tiles (bound by the
// matrix cores) and rests (bound by the weights' stream) alternate, which
// measured 13 % faster than all whole tiles first.  Found by one scan over
// the slots (S <= 1024) in LDS.
template <int BQ, int THREADS>
__device__ __forceinline__ bool find_tile(const RowMap& m, int index, int& slot, int& q0, int& nq) {
    __shared__ int wsum[THREADS / 64], found[3];
    constexpr int PER = 1024 / THREADS;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int2 r[PER];
    int tiles = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int s = t * PER + j;
        r[j] = s < m.S ? slot_range(m, s) : make_int2(0, 0);
        tiles += (r[j].y + BQ - 1) / BQ;
    }
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(sum, o, 64);
        if (lane >= o) sum += x;
    }
    if (lane == 63) wsum[wave] = sum;
    if (t == 0) found[0] = -1;
    __syncthreads();
    sum -= tiles;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w)
        if (w < wave) sum += wsum[w];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int n = (r[j].y + BQ - 1) / BQ, at = index - sum;
        if (at >= 0 && at < n) {
            found[0] = t * PER + j;
            found[1] = r[j].x + at * BQ;
            found[2] = min(BQ, r[j].y - at * BQ);
        }
        sum += n;
    }
    __syncthreads();
    slot = __builtin_amdgcn_readfirstlane(found[0]);
    q0 = __builtin_amdgcn_readfirstlane(found[1]);
    nq = __builtin_amdgcn_readfirstlane(found[2]);
    return slot >= 0;
}

template <typename C>
__global__ __launch_bounds__(C::THREADS, C::QI * C::PI == 4 ? 2 : 1) void expert_tile_kernel(const TileArgs a) {
    // One array for each buffer, so that the compiler can tell the loads into
    // one from the reads of the others.
    __shared__ __attribute__((aligned(16))) uint8_t sq0[C::QBYTES], sq1[C::QBYTES], sp0[C::PBYTES], sp1[C::PBYTES];
    __shared__ int32_t srow[C::MODE == kWeightGrad ? 2 * C::WINDOW : 1];
    TileLds<C> lds;
    lds.q[0] = sq0;
    lds.q[1] = sq1;
    lds.p[0] = sp0;
    lds.p[1] = sp1;
    lds.row[0] = srow;
    lds.row[1] = srow + C::WINDOW;

    const int N = a.N, K = a.K;
    // Groups of neighbouring column tiles of a row tile run on one XCD
    // (workgroup number modulo 8), which serves their rows from its L2; the
    // groups go round the XCDs.
    const int width = C::MODE == kForward ? (C::SWI ? N / 2 : N) : K;  // columns of the output
    const int ptiles = (width + C::COLS - 1) / C::COLS, pgroups = (ptiles + a.group - 1) / a.group;
    const int j = blockIdx.x >> 3, group = j / a.group * 8 + (blockIdx.x & 7), pt = group % pgroups * a.group + j % a.group;
    const int p0 = pt * C::COLS, qt = group / pgroups;
    if (pt >= ptiles) return;
    int slot, q0, nq, c0 = 0, len;
    if (C::MODE == kWeightGrad) {
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
        if (len <= 0) return tile_zero<C>(a, slot, st % ntiles * ptiles + pt, ntiles * ptiles);
        if (len <= C::BK) {
            f32x16 acc[C::QI][C::PI] = {};
            tile_short<C>(a, q0, c0, p0, len, lds, acc);
            return tile_store<C, C::QI>(a, slot, q0, nq, p0, lds, acc);
        }
    } else {
        if (!find_tile<C::BQ, C::THREADS>(a.rows, qt, slot, q0, nq)) return;
        len = C::MODE == kForward ? K : N;
    }
    const int nb = (nq + 32 * C::WQ - 1) / (32 * C::WQ);
    auto body = [&](auto tag) {
        constexpr int NB = decltype(tag)::value;
        f32x16 acc[NB][C::PI] = {};
        tile_product<C, NB>(a, slot, q0, nq, c0, p0, len, lds, acc);
        if constexpr (C::EPI) tile_store_epilogue<C, NB>(a, slot, q0, nq, p0, lds, acc);
        else tile_store<C, NB>(a, slot, q0, nq, p0, lds, acc);
    };
    constexpr int QI = C::QI;
    if (C::MODE == kWeightGrad || nb == QI) body(std::integral_constant<int, QI>{});
    else if (nb == 1) body(std::integral_constant<int, 1>{});
    else if (QI > 2 && nb == 2) body(std::integral_constant<int, QI < 2 ? QI : 2>{});
    else if (QI > 3 && nb == 3) body(std::integral_constant<int, QI < 3 ? QI : 3>{});
}

template <typename C>
static hipError_t tile_launch(const TileArgs& a, hipStream_t s) {
    const int width = C::MODE == kForward ? (C::SWI ? a.N / 2 : a.N) : a.K;
    const long long ptiles = (width + C::COLS - 1) / C::COLS;
    const long long qtiles = C::MODE == kWeightGrad
                                 ? (long long)((a.N + C::BQ - 1) / C::BQ) * a.rows.S * a.splits
                                 : a.rows.R / C::BQ + (a.rows.R < a.rows.S ? a.rows.R : a.rows.S);
    // Few row tiles: groups of four column tiles and less, so that every XCD gets
    // some (512 rows of one 8192 x 4096 matrix: 45 us, 76 with all columns of a
    // row tile on one XCD; 8192 x 8192 x 8192: 821 and 870 us).  Many: up to 16,
    // fewer XCDs then read a row (128 slots of 256 rows, 1536 x 2048: 226 us,
    // 235 with four).
    const long long most = qtiles >= 64 ? 16 : qtiles * ptiles >= 256 ? 4 : 1, groups = (ptiles + most - 1) / most;
    TileArgs t = a;
    t.group = (int)((ptiles + groups - 1) / groups);
    const long long grid = (qtiles * ((ptiles + t.group - 1) / t.group) + 7) / 8 * 8 * t.group;
    if (grid > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    expert_tile_kernel<C><<<dim3((uint32_t)grid), C::THREADS, 0, s>>>(t);
    return hipGetLastError();
}

// 256 x 256 by eight waves of 128 x 64, 128 x 128 by four of 64 x 64.
template <int DT, int MODE, bool SWI, bool EPI = false>
static hipError_t tile_launch_size(const TileArgs& a, int big, hipStream_t s) {
    return big ? tile_launch<Tile<DT, MODE, SWI, 4, 2, 2, 4, EPI>>(a, s)
               : tile_launch<Tile<DT, MODE, SWI, 2, 2, 2, 2, EPI>>(a, s);
}

template <int DT>
static hipError_t tile_launch_type(const TileArgs& a, int mode, int act, int big, hipStream_t s) {
    if (mode == kForward) return act ? tile_launch_size<DT, kForward, true>(a, big, s) : tile_launch_size<DT, kForward, false>(a, big, s);
    if (mode == kDataGrad) return tile_launch_size<DT, kDataGrad, false>(a, big, s);
    return tile_launch_size<DT, kWeightGrad, false>(a, big, s);
}

template <int DT>
static hipError_t tile_launch_bias(const TileArgs& a, int act, int big, hipStream_t s) {
    return act ? tile_launch_size<DT, kForward, true, true>(a, big, s) : tile_launch_size<DT, kForward, false, true>(a, big, s);
}

hipError_t launch_tile_bias_bf16(const TileArgs& a, int act, int big, hipStream_t s);
hipError_t launch_tile_bias_f16(const TileArgs& a, int act, int big, hipStream_t s);
hipError_t launch_tile_bf16(const TileArgs& a, int mode, int act, int big, hipStream_t s);
hipError_t launch_tile_f16(const TileArgs& a, int mode, int act, int big, hipStream_t s);

}  // namespace qmoe
