// One tile of a matrix product on the matrix cores (device, internal).
#pragma once

#include "zs_common.h"

namespace zs {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileK = 64;

template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr int kThreads = WM * WN * 64;
    static constexpr int TM = BM / WM, TN = BN / WN;      // a wave's part
    static constexpr int MI = TM / 16, NI = TN / 16;      // fragments of it
    static constexpr int kStage = (BM + BN) * kTileK;   // 16-bit elements
    static constexpr unsigned kLds = STAGES * kStage * 2;
};

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(i16x8 a, i16x8 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) uint16_t Lds16;

// Which rows and columns of a wave's part its fragments stand for.  A lane of a
// result holds one row and four columns of a fragment pair; what they are of the
// whole is free, and chosen so that a lane has MI neighbouring rows and eight
// neighbouring columns: 16-byte accesses along either side in every epilogue.
//   fragment i, lane a (of 16):      row     a MI + i
//   fragment 2 u + v, row 4 g + s:   column  32 u + 8 g + 4 v + s
template <class T>
__device__ __forceinline__ int row_of(int p) {       // p: 16 i + a, of all waves
    return p / T::TM * T::TM + p % 16 * T::MI + p % T::TM / 16;
}
template <class T>
__device__ __forceinline__ int column_of(int p) {    // p: 16 j + 4 g + s
    return p / 32 * 32 + p % 16 / 4 * 8 + p % 32 / 16 * 4 + p % 4;
}

// An operand's place in device memory, k innermost ("rows": X[row][k]) or
// outermost ("columns": X[k][row]).  Its rows (columns) come in blocks of 64, which
// a row-major matrix has 64 rows (64 elements) apart; a matrix in the workspace
// is kept in blocks of 64 x 64, each 8 KiB in one piece (blocked()).
struct Operand {
    const uint16_t* p;
    int64_t pitch;     // elements from one row (k row) to the next
    int64_t block;     // from one block of rows (columns) to the next
    int64_t step;      // from one k tile to the next
    int extent;        // rows (columns form: a multiple of 8)
};
__device__ __forceinline__ Operand by_rows(const uint16_t* p, int64_t pitch, int extent) {
    return Operand{p, pitch, 64 * pitch, kTileK, extent};
}
__device__ __forceinline__ Operand by_columns(const uint16_t* p, int64_t pitch, int extent) {
    return Operand{p, pitch, 64, kTileK * pitch, extent};
}
constexpr int kBlockElems = 64 * 64;
// across: blocks in a row of them
__device__ __forceinline__ Operand blocked_by_rows(const uint16_t* p, int across, int extent) {
    return Operand{p, 64, (int64_t)across * kBlockElems, kBlockElems, extent};
}
__device__ __forceinline__ Operand blocked_by_columns(const uint16_t* p, int across, int extent) {
    return Operand{p, 64, kBlockElems, (int64_t)across * kBlockElems, extent};
}
__host__ __device__ __forceinline__ int64_t blocked(int row, int column, int across) {
    return ((int64_t)(row >> 6) * across + (column >> 6)) * kBlockElems + (row & 63) * 64 + (column & 63);
}

// Device memory straight into LDS: 64 lanes x 16 bytes, lane after lane from
// `lds` (of the whole wave) on.  In asm: of its own loads of this kind the compiler
// does not know which LDS reads they meet, and puts a wait for all of them before
// every transposing read (8192 x 8192 x 8192 with b's columns: 1097 -> 1272
// TFLOP/s).  It does not wait for these at a barrier either: loads_done().
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(from)
                 : "memory");   // M0 is not allocated: the compiler sets it before each use of its own
}
// All loads to LDS of this wave but the last N have arrived (of the other waves': a
// barrier after it).  With N > 0 no other vector memory access may come between.
template <int N>
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

enum Side : int { kA, kB, kBCols };   // the left operand; the right one by rows; by columns

template <class T, int SIDE>
struct Stager {
    static constexpr int ROWS = SIDE == kA ? T::BM : T::BN, THREADS = T::kThreads;
    static constexpr int kChunks = ROWS * kTileK / 8 / THREADS;
    static_assert(kChunks * 8 * THREADS == ROWS * kTileK, "whole rounds of 16-byte chunks");
    uint32_t off[kChunks];   // bytes from the operand's k position
    uint64_t base, step;     // bytes; step per k tile

    // Where a chunk of 8 elements is among its row's in LDS, so that lanes that read
    // together meet no bank twice.
    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (SIDE != kBCols) return (row >> 1) & 7;          // 16 rows of 128 bytes
        else if constexpr (ROWS >= 128) return ((row >> 3) & 1) | (row & 3) << 2;          // rows are k here
        else return ((row >> 3) & 1) | ((row >> 1) & 1) << 2;
    }
    __device__ __forceinline__ void init(const Operand& o, int first) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int p = i * THREADS + (int)threadIdx.x;
            if constexpr (SIDE == kBCols) {
                constexpr int per = ROWS / 8;
                const int k = p / per, c = (p % per) ^ swizzle(k);
                const int at = min(first + c * 8, o.extent - 8) - first;   // past the edge: some column, not used
                off[i] = (uint32_t)((k * o.pitch + (at >> 6) * o.block + (at & 63)) * 2);
            } else {
                const int row = p / 8, c = (p % 8) ^ swizzle(row);
                const int of = SIDE == kA ? row_of<T>(row) : column_of<T>(row);
                const int at = min(first + of, o.extent - 1) - first;
                off[i] = (uint32_t)(((at >> 6) * o.block + (at & 63) * o.pitch + c * 8) * 2);
            }
        }
        base = reinterpret_cast<uint64_t>(o.p + (first >> 6) * o.block);   // (tiles start on blocks)
        step = (uint64_t)o.step * 2;
    }
    // the next k tile to `lds` on; wave0: this wave's first thread
    __device__ __forceinline__ void issue(Lds16* lds, int wave0) {
        const __amdgpu_buffer_rsrc_t from =
            __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, 0xFFFFFFFFu, 0x00027000);
        const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)lds) + wave0 * 16;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            load_to_lds(from, off[i], (uint32_t)__builtin_amdgcn_readfirstlane((int)(at + i * THREADS * 16)));
        base += step;
    }
    // Fragment f of a wave whose part starts at `part`, k from 32 * ks: lane l holds row l % 16 of it, k = 8 (l / 16) ...
    static __device__ __forceinline__ i16x8 fragment(const Lds16* lds, int part, int f, int ks) {
        const int l = threadIdx.x & 63;
        if constexpr (SIDE == kBCols) {
            // 16 lanes transpose 4 k rows of 4 x 4 elements: lane t gives 4 of k row t / 4, and
            // gets 4 k of element t.  In odd groups of columns the halves of a chunk are
            // exchanged (both halves' banks are used then): pair_of() puts them back.
            const int t = l & 15, g = t & 3, c = (part >> 3) + f / 2 * 4 + g, half = (f ^ g) & 1;
            i16x4 h[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = ks * 32 + (l >> 4) * 8 + j * 4 + (t >> 2);
                h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(
                    const_cast<Lds16*>(lds) + k * ROWS + ((c ^ swizzle(k)) << 3) + half * 4));
            }
            return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int r = part + 16 * f + (l & 15), c = ks * 4 + (l >> 4);
            return *(const __attribute__((address_space(3))) i16x8*)(lds + r * kTileK + ((c ^ swizzle(r)) << 3));
        }
    }
};

// acc: a tile's sums (pair_of and lane_place say where).
//
// One k tile in LDS is multiplied while the next STAGES - 1 ones' loads arrive.  Two
// stages of the largest tiles fill most of the LDS; a workgroup of the smallest ones
// waits for little but its loads, and has three.
// A tile is worked through in phases of two rows of fragments; each phase first
// starts the LDS reads of the next one's fragments, so that they arrive behind
// its matrix instructions.  The last phase's are in the next tile: before it
// comes the barrier, and after the barrier the loads of the tile after that,
// which have a whole tile's time.  8192 x 8192 x 8192 in fp16, against reading
// each phase's fragments at its start: 1235 -> 1295 TFLOP/s with b's rows, 1033
// -> 1272 with its columns; with 16-byte stores (row_of, column_of) 1322 and
// 1283 (a library product: 1315, 1249; on zeros, which do not reach the power
// limit, 1585 and 1579).
template <class T, bool BF16, bool BCOLS>
__device__ __forceinline__ void multiply(const Operand& a, const Operand& b, int m0, int n0, int tiles, Lds16* lds,
                                         f32x4 (&acc)[T::MI][T::NI]) {
    Stager<T, kA> sa;
    Stager<T, BCOLS ? kBCols : kB> sb;
    sa.init(a, m0);
    sb.init(b, n0);
    const int wave0 = __builtin_amdgcn_readfirstlane((int)(threadIdx.x & ~63u)), wave = wave0 >> 6;
    const int wm = wave / T::WN * T::TM, wn = wave % T::WN * T::TN;
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    if (tiles == 0) return;
    constexpr int kG = T::MI / 2, kPhases = 2 * kG;   // phases of 32 of a tile's 64 k; of all
    constexpr int kAt = T::BM * kTileK, kPer = (T::NI + kG - 1) / kG;
    constexpr int kLoads = sa.kChunks + sb.kChunks;   // of one k tile, by a wave
    constexpr int kMore = (T::STAGES - 2) * kLoads;   // that may be under way when the next tile is needed
    auto stage = [&](int t) { return lds + t % T::STAGES * T::kStage; };
    auto issue = [&](int t) {
        Lds16* const to = stage(t);
        sa.issue(to, wave0);
        sb.issue(to + kAt, wave0);
    };
    issue(0);
    loads_done<0>();
    __syncthreads();
#pragma unroll
    for (int t = 1; t < T::STAGES; ++t)
        if (t < tiles) issue(t);
    Lds16 *cur = lds, *next = stage(1);
    i16x8 fa[2][2], fb[2][T::NI];
#pragma unroll
    for (int j = 0; j < T::NI; ++j) fb[0][j] = sb.fragment(cur + kAt, wn, j, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) fa[0][i] = sa.fragment(cur, wm, i, 0);
    for (int t = 0; t < tiles; ++t) {
#pragma unroll
        for (int q = 0; q < kPhases; ++q) {
            const int ks = q / kG, g = q % kG;
            if (q == kPhases - 1) {
                // (with fewer tiles left than stages, fewer loads are under way)
                if (kMore > 0 && t + T::STAGES <= tiles) loads_done<kMore>();
                else loads_done<0>();
                __syncthreads();
                if (t + T::STAGES < tiles) issue(t + T::STAGES);
                // (past the last tile: what the other buffer held, not used)
#pragma unroll
                for (int i = 0; i < 2; ++i) fa[(q + 1) & 1][i] = sa.fragment(next, wm, i, 0);
#pragma unroll
                for (int j = 0; j < T::NI; ++j) fb[0][j] = sb.fragment(next + kAt, wn, j, 0);
            } else {
                const int s = (q + 1) / kG, h = (q + 1) % kG;
#pragma unroll
                for (int i = 0; i < 2; ++i) fa[(q + 1) & 1][i] = sa.fragment(cur, wm, 2 * h + i, s);
                if (ks == 0) {
#pragma unroll
                    for (int j = g * kPer; j < (g + 1) * kPer && j < T::NI; ++j) fb[1][j] = sb.fragment(cur + kAt, wn, j, 1);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < T::NI; ++j) acc[2 * g + i][j] = mfma<BF16>(fb[ks][j], fa[q & 1][i], acc[2 * g + i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        cur = next;
        next = T::STAGES == 2 ? stage(t) : stage(t + 2);
    }
    __syncthreads();   // the LDS is the caller's again
}

// The eight neighbouring columns that fragments 2 u and 2 u + 1 hold of row i.
template <class T, bool BCOLS>
__device__ __forceinline__ void pair_of(const f32x4 (&acc)[T::MI][T::NI], int i, int u, f32x4 (&x)[2]) {
    const f32x4 first = acc[i][2 * u], second = acc[i][2 * u + 1];
    const bool exchanged = BCOLS && (threadIdx.x & 16) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {   // (a choice of values, not of addresses: acc stays in registers)
        x[0][k] = exchanged ? second[k] : first[k];
        x[1][k] = exchanged ? first[k] : second[k];
    }
}
// This lane's first row and first column of a tile at (m0, n0); the rows are MI
// neighbours, the columns eight of every 32.
template <class T>
__device__ __forceinline__ void lane_place(int m0, int n0, int& row, int& column) {
    const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    row = m0 + wave / T::WN * T::TM + (l & 15) * T::MI;
    column = n0 + wave % T::WN * T::TN + (l >> 4) * 8;
}

}  // namespace zs
