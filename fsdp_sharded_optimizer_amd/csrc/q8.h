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

// the dither word of the first of 4 consecutive elements (the group G = i / 4
// of its tensor); the j-th's is j * kGolden more
__device__ __forceinline__ uint32_t q8_word(uint64_t group, uint32_t tensor_key) {
    return q8_mix((uint32_t)group + (uint32_t)(group >> 32) * kGolden + tensor_key);
}

// Largest of the 64 lanes' values, in every lane.  DPP within the wave: shifts
// inside the 16-lane rows, then the two broadcasts across them; lane 63 has
// the result.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
    return x > y ? x : y;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = dpp_max<0x111, 0xF>(x);   // row_shr:1
    x = dpp_max<0x112, 0xF>(x);
    x = dpp_max<0x114, 0xF>(x);
    x = dpp_max<0x118, 0xF>(x);
    x = dpp_max<0x142, 0xA>(x);   // row_bcast:15
    x = dpp_max<0x143, 0xC>(x);   // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max4(const float (&x)[4]) {
    const uint32_t a = magnitude(x[0]), b = magnitude(x[1]), c = magnitude(x[2]), d = magnitude(x[3]);
    const uint32_t p = a > b ? a : b, q = c > d ? c : d;
    return p > q ? p : q;
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
    constexpr uint32_t kMask = TOP == kTopM ? 0x87F00000u : 0x0FF00000u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // exp_avg: the code's sign, extended, ends in bit 31; its 7 other bits in 26..20
        const uint32_t at20 = TOP == kTopM ? (uint32_t)((int32_t)(codes << (24 - 8 * j)) >> 4)
                                           : (j < 3 ? codes << (20 - 8 * j) : codes >> 4);
        x[j] = __uint_as_float(at20 & kMask);
    }
}

// The values of 4 codes in a word; e: their block's scale byte.
template <int TOP>
__device__ __forceinline__ void q8_decode4(uint32_t codes, uint32_t e, float (&x)[4]) {
    q8_unpack4<TOP>(codes, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = e == 255u ? __builtin_nanf("") : __builtin_ldexpf(x[j], (int)e - TOP);
}

// 4 values into codes; word: the dither word of the first.  The sum cannot
// carry past the top code: the block's largest magnitude is at most 1.875 times
// the top exponent's power of two, which is the top code.  (In a block with
// e = 255 nothing of a code is meaningful; it is only kept inside its byte.)
template <int TOP>
__device__ __forceinline__ uint32_t q8_encode4(const float (&x)[4], uint32_t e, uint32_t word) {
    uint32_t c[4];   // the code in the top byte
    if (plain_scale<TOP>(e)) {
        const float scale = exp2_of(TOP - (int)e);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(x[j] * scale);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(__builtin_ldexpf(x[j], TOP - (int)e));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t h = word + (uint32_t)j * kGolden;
        const uint32_t sum = c[j] + (TOP == kTopM ? h >> 12 : h & 0xFFFFFu);
        if constexpr (TOP == kTopM) c[j] = ((sum << 4) & 0x7FFFFFFFu) | (sum & 0x80000000u);
        else c[j] = sum << 4;
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
    const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0703u);   // top bytes of c[0], c[1]
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x07030C0Cu), lo, 0x07060100u);
}

// Where a tensor's (entry's) codes and scales are.  Codes lie in chunks of
// kQ8Pad elements: the code of element 256 b + 4 l + j of a chunk (block b,
// lane l) is its byte 16 l + 4 b + j, so a lane's codes of all four blocks are one
// 128-bit access, and every stream of a wave is lane-contiguous.
struct Q8At {
    uint8_t* m;
    uint8_t* v;
    uint8_t* scales;   // two bytes per block: exp_avg's, exp_avg_sq's
};
__device__ __forceinline__ Q8At q8_at(const Q8Entry& e) {
    const int64_t off = (int64_t)e.off * kQ8Pad, padded = (int64_t)e.padded * kQ8Pad;
    return Q8At{e.state + off, e.state + padded + off, e.state + 2 * padded + off / (kQ8Block / 2)};
}

}  // namespace zs
