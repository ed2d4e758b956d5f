// One tile of a matrix product on the matrix cores (device, internal).
#pragma once

#include "zs_common.h"

namespace zs {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileK = 64;

template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = WM * WN * 64;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    static constexpr int kStage = (BM + BN) * kTileK;   // 16-bit elements
    static constexpr unsigned kLds = 2 * kStage * 2;
};

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(i16x8 a, i16x8 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) uint16_t Lds16;

// An operand's place in device memory, k innermost ("rows": X[row][k]) or
// outermost ("columns": X[k][row]).
struct Operand {
    const uint16_t* p;
    int64_t pitch;     // elements
    int extent;        // rows (columns form: a multiple of 8)
};

template <int ROWS, int THREADS, bool COLS>
struct Stager {
    static constexpr int kChunks = ROWS * kTileK / 8 / THREADS;
    static_assert(kChunks * 8 * THREADS == ROWS * kTileK, "whole rounds of 16-byte chunks");
    uint32_t off[kChunks];   // bytes from the operand's k position
    const char* base;
    int64_t step;            // bytes per k tile

    static __device__ __forceinline__ int swizzle(int k) {   // of a k row of the columns form, in chunks
        if constexpr (ROWS >= 128) return 2 * ((k & 3) | ((k >> 3) & 1) << 2);
        else return 2 * (((k >> 1) & 1) | ((k >> 3) & 1) << 1);
    }
    __device__ __forceinline__ void init(const Operand& o, int first) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int p = i * THREADS + (int)threadIdx.x;
            if constexpr (COLS) {
                constexpr int per = ROWS / 8;
                const int k = p / per, c = (p % per) ^ swizzle(k);
                const int at = min(first + c * 8, o.extent - 8) - first;   // past the edge: some column, not used
                off[i] = (uint32_t)(((int64_t)k * o.pitch + at) * 2);
            } else {
                const int row = p / 8, c = (p % 8) ^ ((row >> 1) & 7);
                const int at = min(first + row, o.extent - 1) - first;
                off[i] = (uint32_t)(((int64_t)at * o.pitch + c * 8) * 2);
            }
        }
        if constexpr (COLS) {
            base = reinterpret_cast<const char*>(o.p + first);
            step = o.pitch * kTileK * 2;
        } else {
            base = reinterpret_cast<const char*>(o.p + (int64_t)first * o.pitch);
            step = kTileK * 2;
        }
    }
    __device__ __forceinline__ void issue(Lds16* lds) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void*)(base + (int64_t)off[i]),
                (__attribute__((address_space(3))) void*)(lds + (i * THREADS + (threadIdx.x & ~63u)) * 8), 16, 0, 0);
        base += step;
    }
    // the fragment of 16 rows from `row` and k from 32 * ks: lane l holds row l % 16, k = 8 (l / 16) ...
    static __device__ __forceinline__ i16x8 fragment(const Lds16* lds, int row, int ks) {
        const int l = threadIdx.x & 63;
        if constexpr (COLS) {
            // 16 lanes transpose 4 k rows of 16 elements: lane t gives 4 of k row t / 4, and gets 4 k of element t
            const int t = l & 15;
            i16x4 h[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = ks * 32 + (l >> 4) * 8 + j * 4 + (t >> 2);
                const int c = (row >> 3) + ((t >> 1) & 1);
                const int at = k * ROWS + ((c ^ swizzle(k)) << 3) + (t & 1) * 4;
                h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) i16x4*)(const_cast<Lds16*>(lds) + at));
            }
            return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int r = row + (l & 15), c = ks * 4 + (l >> 4);
            return *(const __attribute__((address_space(3))) i16x8*)(lds + r * kTileK + ((c ^ ((r >> 1) & 7)) << 3));
        }
    }
};

// acc[i][j]: rows m = wave row + 16 i + lane % 16, columns n = wave column + 16 j + 4 (lane / 16) + 0..3
template <class T, bool BF16, bool BCOLS>
__device__ __forceinline__ void multiply(const Operand& a, const Operand& b, int m0, int n0, int tiles, Lds16* lds,
                                         f32x4 (&acc)[T::MI][T::NI]) {
    Stager<T::BM, T::kThreads, false> sa;
    Stager<T::BN, T::kThreads, BCOLS> sb;
    sa.init(a, m0);
    sb.init(b, n0);
    const int wave = threadIdx.x >> 6, wm = (wave / T::WN) * (T::BM / T::WM), wn = (wave % T::WN) * (T::BN / T::WN);
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    if (tiles == 0) return;
    sa.issue(lds);
    sb.issue(lds + T::BM * kTileK);
    __syncthreads();
    Lds16 *cur = lds, *next = lds + T::kStage;
    for (int t = 0; t < tiles; ++t) {
        if (t + 1 < tiles) {
            sa.issue(next);
            sb.issue(next + T::BM * kTileK);
        }
#pragma unroll
        for (int ks = 0; ks < kTileK / 32; ++ks) {
            i16x8 fa[T::MI], fb[T::NI];
#pragma unroll
            for (int j = 0; j < T::NI; ++j) fb[j] = sb.fragment(cur + T::BM * kTileK, wn + 16 * j, ks);
#pragma unroll
            for (int i = 0; i < T::MI; ++i) fa[i] = sa.fragment(cur, wm + 16 * i, ks);
#pragma unroll
            for (int i = 0; i < T::MI; ++i)
#pragma unroll
                for (int j = 0; j < T::NI; ++j) acc[i][j] = mfma<BF16>(fb[j], fa[i], acc[i][j]);
        }
        __syncthreads();
        Lds16* const x = cur;
        cur = next;
        next = x;
    }
}

}  // namespace zs
