// One tile of a gradient in a workgroup's squared norm (device, internal).
#pragma once

#include "reduce.h"
#include "tensors.h"

namespace zs {
namespace {

constexpr int kNormQ = 4;
constexpr unsigned kNormLds = 24576;
template <bool BF16> constexpr int kNormVec = BF16 ? 8 : 4;   // elements of a 128-bit load
template <bool BF16> constexpr int64_t kNormTile = (int64_t)kBlock * kNormVec<BF16> * kNormQ;

// the elements from `at` of n that a 128-bit load would bring, zeros past the end
template <bool BF16>
__device__ __forceinline__ u32x4 last_words(const typename GradType<BF16>::T* grad, int at, int n) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (BF16)
            w[j] = (at + 2 * j < n ? (uint32_t)grad[at + 2 * j] : 0u) |
                   (at + 2 * j + 1 < n ? (uint32_t)grad[at + 2 * j + 1] << 16 : 0u);
        else
            w[j] = at + j < n ? __float_as_uint(grad[at + j]) : 0u;
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}

// This thread's share of a tile's sum of squares.  n: the tile's elements; last: it
// may be a ragged one; odd: a bf16 gradient at an odd element offset.
template <bool BF16, bool KEEP>
__device__ __forceinline__ double norm_tile(const typename GradType<BF16>::T* grad, int n, bool last, bool odd, float scale) {
    constexpr int VE = kNormVec<BF16>;
    const int lane0 = threadIdx.x * VE;
    u32x4 v[kNormQ];
    if (BF16 && odd && !last) {
        // bf16 at an odd offset: a lane's 16 bytes would span 5 words.  The words
        // from its second element on instead; its first element is in the last
        // word of the lane before (of a wave's first lane: loaded by itself).
        uint32_t head[kNormQ] = {};
#pragma unroll
        for (int q = 0; q < kNormQ; ++q) v[q] = ld_u32x4_any<KEEP>(grad + lane0 + q * kBlock * VE + 1);
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int q = 0; q < kNormQ; ++q) head[q] = (uint32_t)grad[lane0 + q * kBlock * VE] << 16;
        }
#pragma unroll
        for (int q = 0; q < kNormQ; ++q) {
            const u32x4 w = v[q];
            const uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp((int)head[q], (int)w.w, 0x138, 0xF, 0xF, false);   // wave_shr:1
            v[q] = u32x4{__builtin_amdgcn_alignbit(w.x, before, 16), __builtin_amdgcn_alignbit(w.y, w.x, 16),
                         __builtin_amdgcn_alignbit(w.z, w.y, 16), __builtin_amdgcn_alignbit(w.w, w.z, 16)};
        }
    } else if (n == (int)kNormTile<BF16>) {
#pragma unroll
        for (int q = 0; q < kNormQ; ++q) v[q] = ld_u32x4_any<KEEP>(grad + lane0 + q * kBlock * VE);
    } else {   // a tensor's ragged last tile: elements past the end add +0
#pragma unroll
        for (int q = 0; q < kNormQ; ++q) {
            const int at = lane0 + q * kBlock * VE;
            if (at + VE <= n) v[q] = ld_u32x4_any<KEEP>(grad + at);
            else v[q] = last_words<BF16>(grad, at, n);
        }
    }
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int q = 0; q < kNormQ; ++q) {
        if constexpr (BF16) {
            const float lo[4] = {bf16_to_f32(v[q].x & 0xFFFFu), bf16_to_f32(v[q].x >> 16),
                                 bf16_to_f32(v[q].y & 0xFFFFu), bf16_to_f32(v[q].y >> 16)};
            const float hi[4] = {bf16_to_f32(v[q].z & 0xFFFFu), bf16_to_f32(v[q].z >> 16),
                                 bf16_to_f32(v[q].w & 0xFFFFu), bf16_to_f32(v[q].w >> 16)};
            add_squares4(lo, scale, s0, s1);
            add_squares4(hi, scale, s0, s1);
        } else {
            const float g[4] = {__uint_as_float(v[q].x), __uint_as_float(v[q].y), __uint_as_float(v[q].z),
                                __uint_as_float(v[q].w)};
            add_squares4(g, scale, s0, s1);
        }
    }
    return s0 + s1;
}

}  // namespace
}  // namespace zs
