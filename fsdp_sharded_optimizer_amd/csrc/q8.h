// 8-bit moments (device): the codes, their scales and the dither, as
// include/zshard_tensors.h defines them (internal).
#pragma once

#include "tensors.h"

namespace zs {

constexpr int kTopM = 15;   // exponent field of the largest codes: 4 bits for exp_avg,
constexpr int kTopV = 31;   // 5 for exp_avg_sq
constexpr uint32_t kGolden = 0x9E3779B9u;

__host__ __device__ __forceinline__ uint32_t q8_mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

// the dither word of the first element of the group G = i / 4 of a tensor,
// before its mixing (the mixed word's j-th element's is j * kGolden more)
__device__ __forceinline__ uint32_t q8_group(uint64_t group, uint32_t tensor_key) {
    return (uint32_t)group + (uint32_t)(group >> 32) * kGolden + tensor_key;
}

// The largest of the 64 lanes' values, for 4 values at once: x[k]'s result ends
// in lane max_lane(k).  Each step halves the registers while it reduces: after
// exchanging the halves (rows) of two registers, one maximum reduces both.  10
// operations in all, against 6 for each value by itself.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {   // lanes 0-31: a, 32-63: b
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    return max2(r[0], r[1]);
}
__device__ __forceinline__ uint32_t max_rows(uint32_t a, uint32_t b) {     // rows 0, 2: a, rows 1, 3: b
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    return max2(r[0], r[1]);
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {   // CTRL: a permutation of the lanes
    return max2(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(const uint32_t (&x)[4]) {
    uint32_t y = dpp_max<0x128>(max_rows(max_halves(x[0], x[1]), max_halves(x[2], x[3])));   // row_ror:8
    y = dpp_max<0xB1>(y);      // quad_perm 1,0,3,2
    y = dpp_max<0x4E>(y);      // quad_perm 2,3,0,1
    return dpp_max<0x141>(y);  // row_half_mirror
}
__device__ constexpr int max_lane(int k) { return (k & 1) * 32 + (k & 2) * 8; }

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max4(const float (&x)[4]) {
    return max2(max2(magnitude(x[0]), magnitude(x[1])), max2(magnitude(x[2]), magnitude(x[3])));
}
// a block's scale byte from its largest magnitude's pattern (NaN patterns are
// above infinity's, so a non-finite block gets 255)
__device__ __forceinline__ uint32_t q8_scale(uint32_t most) {
    const uint32_t e = (most + 0x0FFFFFu) >> 23;
    return e < 255u ? e : 255u;   // the largest NaN patterns carry further
}

// 2^k, -126 <= k <= 127
__device__ __forceinline__ float exp2_of(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// A scale byte whose powers of two 2^(e - TOP) and 2^(TOP - e) are normal
// binary32 numbers, so that scaling is one multiplication: all blocks but those
// whose largest moment is below 2^-112 (exp_avg_sq: 2^-96) or from 2^15 (2^31) up.
template <int TOP>
__device__ __forceinline__ bool plain_scale(uint32_t e) { return e >= (uint32_t)TOP && e <= (uint32_t)TOP + 126u; }

// The 4 codes of a word as binary32 numbers below their scale: value * 2^(TOP - e).
template <int TOP>
__device__ __forceinline__ void q8_unpack4(uint32_t codes, float (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // exp_avg: the code's sign, extended, ends in bit 31; its 7 other bits in 26..20
        if constexpr (TOP == kTopM)
            x[j] = __uint_as_float(((uint32_t)__builtin_amdgcn_sbfe((int)codes, 8 * j, 8) << 20) & 0x87F00000u);
        else
            x[j] = __uint_as_float(__builtin_amdgcn_ubfe(codes, 8 * j, 8) << 20);
    }
}

// Unpacked codes into values; e: their block's scale byte.
template <int TOP>
__device__ __forceinline__ void q8_scale4(uint32_t e, float (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = e == 255u ? __builtin_nanf("") : __builtin_ldexpf(x[j], (int)e - TOP);
}
template <int TOP>
__device__ __forceinline__ void q8_decode4(uint32_t codes, uint32_t e, float (&x)[4]) {
    q8_unpack4<TOP>(codes, x);
    if (plain_scale<TOP>(e)) {
        const float scale = exp2_of((int)e - TOP);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = x[j] * scale;
    } else {
        q8_scale4<TOP>(e, x);
    }
}

// the top bytes of four words, the first one's lowest
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0703u);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x07030C0Cu), lo, 0x07060100u);
}

// 4 values into codes; word: the dither word of the first.  The sum cannot
// carry past the top code: the block's largest magnitude is at most 1.875 times
// the top exponent's power of two, which is the top code.  (In a block with
// e = 255 nothing of a code is meaningful; it is only kept inside its byte.)
template <int TOP>
__device__ __forceinline__ uint32_t q8_encode4(const float (&x)[4], uint32_t e, uint32_t word) {
    uint32_t c[4];   // the code (exp_avg: without its sign) in the top byte
    if (plain_scale<TOP>(e)) {
        const float scale = exp2_of(TOP - (int)e);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(__builtin_fabsf(x[j]) * scale);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = magnitude(__builtin_ldexpf(x[j], TOP - (int)e));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t h = word + (uint32_t)j * kGolden;
        c[j] = (c[j] + (TOP == kTopM ? h >> 12 : h & 0xFFFFFu)) << 4;
    }
    if constexpr (TOP == kTopV) {
        // a positive second moment never becomes 0 (few do: one test for the four)
        const uint32_t least = min(min(c[0], c[1]), min(c[2], c[3]));
        if (least < 0x01000000u) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c[j] < 0x01000000u && x[j] > 0.0f) c[j] = 0x01000000u;
        }
    }
    const uint32_t out = top_bytes(c[0], c[1], c[2], c[3]);
    if constexpr (TOP == kTopV) return out;
    const uint32_t signs = top_bytes(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                     __float_as_uint(x[3]));
    return (signs & 0x80808080u) | (out & 0x7F7F7F7Fu);
}

// Codes lie in chunks of kQ8Pad = 512 elements, a chunk's exp_avg codes and then
// its exp_avg_sq codes: the code of element 256 b + 4 l + j of a chunk (block b,
// lane l) is byte 8 l + 4 b + j of either, so a lane's codes of both blocks are
// one access and every stream of a wave is lane-contiguous.  (Both kinds in one
// run: the step 0.3-1 % faster than in two arrays.)

}  // namespace zs
