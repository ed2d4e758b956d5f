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
__device__ __forceinline__ uint32_t q8_scale(uint32_t most) { return (most + 0x0FFFFFu) >> 23; }

// The values of 4 codes in a word; e: their block's scale byte.
template <int TOP>
__device__ __forceinline__ void q8_decode4(uint32_t codes, uint32_t e, float (&x)[4]) {
    if (e == 255u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __builtin_nanf("");
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t c = (codes >> (8 * j)) & 0xFFu;
        uint32_t bits;
        if constexpr (TOP == kTopM) bits = ((c & 0x7Fu) << 20) | ((c & 0x80u) << 24);
        else bits = c << 20;
        x[j] = __builtin_ldexpf(__uint_as_float(bits), (int)e - TOP);
    }
}

// 4 values into codes; word: the dither word of the first.  The sum cannot
// carry past the top code: the block's largest magnitude is at most 1.875 times
// the top exponent's power of two, which is the top code.  (In a block with
// e = 255 nothing of a code is meaningful; it is only kept inside its byte.)
template <int TOP>
__device__ __forceinline__ uint32_t q8_encode4(const float (&x)[4], uint32_t e, uint32_t word) {
    uint32_t out = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t h = word + (uint32_t)j * kGolden;
        const uint32_t r = TOP == kTopM ? h >> 12 : h & 0xFFFFFu;
        const float s = __builtin_ldexpf(__uint_as_float(magnitude(x[j])), TOP - (int)e);
        uint32_t c = (__float_as_uint(s) + r) >> 20;
        if constexpr (TOP == kTopM) {
            c = (c & 0x7Fu) | ((__float_as_uint(x[j]) >> 31) << 7);
        } else {
            c &= 0xFFu;
            if (c == 0 && x[j] > 0.0f) c = 1;
        }
        out |= c << (8 * j);
    }
    return out;
}

// Where a tensor's (entry's) codes and scales are: element i of the entry,
// block (off + i) / kQ8Block of the tensor.
struct Q8At {
    uint8_t* m;
    uint8_t* v;
    uint8_t* scales;   // two bytes per block
};
__device__ __forceinline__ Q8At q8_at(const Q8Entry& e) {
    const int64_t off = (int64_t)e.off * kQ8Pad, padded = (int64_t)e.padded * kQ8Pad;
    return Q8At{e.state + off, e.state + padded + off, e.state + 2 * padded + off / (kQ8Block / 2)};
}

}  // namespace zs
