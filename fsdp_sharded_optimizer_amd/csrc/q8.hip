// AdamW over a list of tensors with 8-bit moments, and the conversions of
// such moments.
//
// The step decodes a block's moments, forms the new ones as the fp32 step does
// (the operations and roundings of adamw_math.h: codes hang on their last
// bits), updates the parameter, takes the block's two new scales from the
// largest magnitudes and stores the codes: 4 bytes of moments per element
// (read and written) instead of 16.
//
// A wave takes one chunk of kQ8Pad = 512 elements, 2 blocks, 8 elements per lane:
// what a wave does once (finding its tensor, the clip coefficient in binary64)
// is then spread over 8 elements.  With 1024 elements per wave the step is as
// fast over hundreds of millions of elements and 5-15 % slower up to 34M, whose
// launches are only a few waves deep; with 256, 1.5 times slower.
#include "adamw_math.h"
#include "q8.h"

namespace zs {
namespace {

constexpr int kWave = 64;
constexpr int kBlocks = (int)(kQ8Pad / kQ8Block);   // per chunk
// LDS reserved (never touched) per workgroup to cap how many share a CU: too
// many keep too many DRAM rows open.  % of the 8 TB/s peak at 0-5 (32 waves per
// CU, all it takes) / 6 / 7 / 8 / 9 / 11 / 12 KiB: the step on 809M fp32 parameters
// (bf16 gradients, re-casts) 74.3 / 76.7 / 77.5 / 78.9 / 79.8 / 79.0 / 75.7; on 855M
// bf16 parameters 79.7 / 80.7 / 81.4 / 79.5 / 77.4 / 73.3 / 67.1; reading 855M moments
// out 80.7 / 81.4 / 79.4 / 73.4 / 67.6 / 60.4 / 53.8; storing 406M bf16 moments 80.2 /
// 77.6 / 75.1 / 71.5 / 67.6 / 61.4 / 54.8, fp32 ones 79.0 / 79.1 / 79.3 / 79.8 / 81.1 /
// 81.4 / 77.2.  Tiles in runs, on 405M at odd offsets:
// fp32 parameters 66 / 68 / 68 / 67 / 68 / 71 / 72 and 69 at 14, bf16 ones 74 / 76 / 75 / 71 /
// 71 / 68 / 63, reading out 63 / 67 / 71 / 67 / 64 / 58 / 53.
// (2 or 4 waves per workgroup: 0.5-4 points slower; plain instead of streaming
// code accesses: the step 1 point slower.)  Launches of fewer than 2^25 elements
// are not long enough for a cap to help: one tensor of 8M / 16M / 32M / 64M, us
// uncapped and capped, the step on bf16 parameters 16.6, 17.2 / 30.4, 30.7 / 53.2,
// 54.0 / 99.3, 99.9, on fp32 ones 21.0, 21.8 / 38.6, 40.1 / 70.6, 72.2 / 135, 136,
// reading out into bf16 14.0, 14.4 / 21.3, 21.0 / 36.0, 35.8 / 65.1, 63.2, storing
// fp32 moments 15.7, 17.0 / 28.2, 29.7 / 53.6, 54.7 / 107, 101.
template <bool PBF16, bool RUNS> constexpr unsigned kStepLds = PBF16 ? (RUNS ? 6144 : 7168) : (RUNS ? 12288 : 9216);
constexpr unsigned kDecodeLds = 6144, kDecodeRunsLds = 7168;
constexpr unsigned kEncodeLds = 11264;   // of fp32 moments
constexpr int64_t kCapElems = int64_t(1) << 25;
unsigned cap(unsigned lds, int64_t elems) { return elems < kCapElems ? 0 : lds; }

// Where a wave works: its chunk of its tensor.
struct Chunk {
    Q8Entry e;
    uint32_t top, has;
    int64_t entry;     // elements of the tensor's record before the chunk
    uint64_t first;    // of the tensor before it
    int n;             // elements in it
    uint32_t index;    // the tensor's place in the caller's list
    uint8_t* codes;    // the lane's exp_avg codes
    uint8_t* scales;   // the chunk's

    // the j-th pointer's elements of the chunk
    template <typename T>
    __device__ __forceinline__ T* at(int j) const {
        return base<T>(j) + entry;
    }
    template <typename T>
    __device__ __forceinline__ T* base(int j) const {
        return unpack_ptr<T>(e.lo[j], (e.hi >> (8 * j) & 0xFFu) | (top >> (8 * j) & 0xFFu) << 8);
    }
};
__device__ __forceinline__ Chunk chunk_of(const Q8Batch& b, bool runs) {
    const uint32_t w = runs ? tile_in_runs(blockIdx.x, gridDim.x) : blockIdx.x;
    uint32_t first_tile;
    const uint32_t t = find_tensor(b.tab, w, first_tile);
    const uint32_t next = b.tab.start[t + 1], tail = b.tail[t / 2] >> (16 * (t % 2));
    Chunk c;
    c.e = b.e[t];
    c.top = b.top;
    c.has = tail;
    c.entry = (int64_t)(w - first_tile) * kQ8Pad;
    c.first = (uint64_t)b.off * kLaunchElems + (uint64_t)c.entry;
    c.n = w + 1 == next ? (int)(tail & kQ8Tail) + 1 : (int)kQ8Pad;
    c.index = b.index + t;
    const int64_t padded = (int64_t)(b.padded != 0 ? b.padded : next - first_tile) * kQ8Pad;
    uint8_t* const state = c.base<uint8_t>(2);
    c.codes = state + 2 * c.first + threadIdx.x * (4 * kBlocks);
    c.scales = state + 2 * padded + c.first / (kQ8Block / 2);
    return c;
}

// 4 consecutive elements from i of n (zeros past the end).
template <bool KEEP, typename T>
__device__ __forceinline__ void load4(const T* p, int i, int n, bool whole, float (&x)[4]) {
    if (whole || i + 4 <= n) {
        const f32x4 w = ld4<KEEP>(p + i);
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = i + j < n ? widen(p[i + j]) : 0.0f;
    }
}
// fp32 to bf16 by the hardware's conversion, to nearest even (a NaN stays one)
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void st4_hw(float* p, const f32x4& x) { st4(p, x); }
__device__ __forceinline__ void st4_hw(uint16_t* p, const f32x4& x) {
    const u32x2 w = __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4));
    __builtin_nontemporal_store(u32x2_any(w), reinterpret_cast<u32x2_any*>(p));
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int i, int n, bool whole, const float (&x)[4]) {
    if (whole || i + 4 <= n) {
        st4_hw(p + i, f32x4{x[0], x[1], x[2], x[3]});
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) st1(p + i + j, x[j]);
    }
}
static_assert(kBlocks == 2, "two words of codes per lane");
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[kBlocks]) {
    const u32x2 x = ld_stream(reinterpret_cast<const u32x2*>(p));
    w[0] = x.x, w[1] = x.y;
}
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[kBlocks]) {
    st_stream(reinterpret_cast<u32x2*>(p), u32x2{w[0], w[1]});
}

// Until every load of the wave has come: a wave that reads all it needs before it
// writes anything lets DRAM turn from reads to writes less often (reading 855M
// moments out: 77.5 % of the HBM peak without, 80.2 % with).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }   // vmcnt(0)

// A chunk's scale bytes as a word: block b's exp_avg byte and exp_avg_sq byte are
// the bytes 2b and 2b + 1.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
    return *reinterpret_cast<const uint32_t*>(p);
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ uint32_t scale_m(uint32_t s, int b) { return (s >> (16 * b)) & 0xFFu; }
__device__ __forceinline__ uint32_t scale_v(uint32_t s, int b) { return (s >> (16 * b + 8)) & 0xFFu; }

// Stores the moments of a wave's chunk: the blocks' scales from their largest
// magnitudes, then the codes.
__device__ __forceinline__ void store_moments(const Chunk& c, uint32_t key, const float (&m)[kBlocks][4],
                                              const float (&v)[kBlocks][4]) {
    uint32_t most[2 * kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) most[2 * b] = max4(m[b]), most[2 * b + 1] = max4(v[b]);
    const uint32_t e = q8_scale(wave_max(most));
    const uint32_t tensor_key = q8_mix(key + c.index * kGolden);
    // the wave's first group; its groups share the upper 32 bits
    const uint32_t group = q8_group(c.first / 4, tensor_key);
    uint32_t mc[kBlocks], vc[kBlocks], scales = 0;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const uint32_t em = (uint32_t)__builtin_amdgcn_readlane((int)e, max_lane(2 * b));
        const uint32_t ev = (uint32_t)__builtin_amdgcn_readlane((int)e, max_lane(2 * b + 1));
        const uint32_t word = q8_mix(group + b * (uint32_t)(kQ8Block / 4) + threadIdx.x);
        mc[b] = q8_encode4<kTopM>(m[b], em, word);
        vc[b] = q8_encode4<kTopV>(v[b], ev, word);
        scales |= (em | ev << 8) << (16 * b);
    }
    store_codes(c.codes, mc);
    store_codes(c.codes + kQ8Pad, vc);
    if (threadIdx.x == 0) *reinterpret_cast<uint32_t*>(c.scales) = scales;
}

// u / step_size of one element from its new moments
template <bool FAST>
__device__ __forceinline__ float adam_ratio(const AdamwScalars& a, float inv_root, float m, float v) {
    if constexpr (FAST) {
        // The hardware's square root and reciprocal are within 1 ulp (2^-23 of
        // the value), the sum and the product half of one: u is within 8 * 2^-24
        // of the exact quotient, far below the parameter's own rounding, for 11
        // issue slots against about 50 for IEEE division and root.
        const float den = __builtin_fmaf(__builtin_amdgcn_sqrtf(v), inv_root, a.eps);
        return m * __builtin_amdgcn_rcpf(den);
    }
    float den = sqrtf(v) / a.bias_correction2_sqrt;
    den = den + a.eps;
    return m / den;
}
// Whether adam_ratio<true>'s bound holds: the hardware's instructions flush
// subnormals.  A subnormal v loses its root, below 2^-63: at most 2^-63 /
// (bias_correction2_sqrt * eps) of den, which at 2^-40 and more is 2 * 2^-24, with
// the 3 * 2^-24 of reciprocal and product under 8.  A den above 2^126 loses its
// reciprocal, and all of it but eps is below 2^100 (a root up to 2^64, over a
// correction of 2^-27 or more).  By the exponents alone, which are scalar
// instructions: the product of two numbers is at least that of their powers of two.
__device__ __forceinline__ bool fast_ratio(const AdamwScalars& a) {
    const uint32_t eps = __float_as_uint(a.eps) >> 23, root = __float_as_uint(a.bias_correction2_sqrt) >> 23;
    return eps + root >= 2 * 127 - 40 && eps < 127 + 100;
}

// One chunk's step.  WHOLE: all its elements are the tensor's.  KEEP: of the
// gradients (keep_grads).  RUNS: the written streams lie off cache lines, tiles are
// taken in runs, and a parameter line that two tiles share is kept in their L2
// (405M fp32 parameters at odd offsets 1210 -> 1184 us, bf16 727 -> 714; on aligned
// tensors 1-4 % slower).
template <bool PBF16, bool GBF16, bool WHOLE, bool FAST, bool KEEP, bool RUNS>
__device__ __forceinline__ void step_chunk(const Q8Batch& b, const Q8Scalars& sc, const Chunk& c) {
    using P = typename GradType<PBF16>::T;
    using G = typename GradType<GBF16>::T;
    const int n = c.n, i = threadIdx.x * 4;
    P* const param = c.at<P>(0);
    const G* const grad = c.at<const G>(1);
    uint16_t* const copy = c.at<uint16_t>(3);
    float g[kBlocks][4], p[kBlocks][4], m[kBlocks][4], v[kBlocks][4];
    uint32_t mc[kBlocks], vc[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) load4<KEEP>(grad, i + k * (int)kQ8Block, n, WHOLE, g[k]);
    load_codes(c.codes, mc);
    load_codes(c.codes + kQ8Pad, vc);
    uint32_t scales = load_scales(c.scales);
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) load4<RUNS>(param, i + k * (int)kQ8Block, n, WHOLE, p[k]);
    float coef;
    if (!clip_coef(sc.adamw, b.norm_sq, coef)) return;
    scales = uniform(scales);
    const AdamwScalars& a = sc.adamw;
    const float inv_root = __builtin_amdgcn_rcpf(a.bias_correction2_sqrt);
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const uint32_t em = scale_m(scales, k), ev = scale_v(scales, k);
        // beta * value: the scale, a power of two, goes into the factor, which
        // changes no bit of the product
        q8_unpack4<kTopM>(mc[k], m[k]);
        q8_unpack4<kTopV>(vc[k], v[k]);
        float keep_m = a.beta1 * exp2_of((int)em - kTopM), keep_v = a.beta2 * exp2_of((int)ev - kTopV);
        if (!plain_scale<kTopM>(em) || !plain_scale<kTopV>(ev)) {
            q8_scale4<kTopM>(em, m[k]);
            q8_scale4<kTopV>(ev, v[k]);
            keep_m = a.beta1;
            keep_v = a.beta2;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) g[k][j] = g[k][j] * a.grad_scale;
        if (coef != 1.0f) {   // (x * 1 is x)
#pragma unroll
            for (int j = 0; j < 4; ++j) g[k][j] = g[k][j] * coef;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gj = g[k][j];
            const float m_keep = keep_m * m[k][j], m_new = a.one_minus_beta1 * gj;
            m[k][j] = m_keep + m_new;
            const float v_keep = keep_v * v[k][j], v_new = a.one_minus_beta2 * (gj * gj);
            v[k][j] = v_keep + v_new;
            p[k][j] = __builtin_fmaf(-adam_ratio<FAST>(a, inv_root, m[k][j], v[k][j]), a.step_size, p[k][j] * a.decay);
            // past the end: no part of the block's scale
            if (!WHOLE && i + k * (int)kQ8Block + j >= n) m[k][j] = v[k][j] = 0.0f;
        }
        store4(param, i + k * (int)kQ8Block, n, WHOLE, p[k]);
        if (!PBF16 && (c.has & kQ8Has3)) store4(copy, i + k * (int)kQ8Block, n, WHOLE, p[k]);
    }
    store_moments(c, sc.key, m, v);
}

template <bool PBF16, bool GBF16, bool DEV, bool KEEP, bool RUNS>
__global__ __launch_bounds__(kWave) void adamw_q8_kernel(const Q8Batch b) {
    const Chunk c = chunk_of(b, RUNS);
    const Q8Scalars sc = DEV ? *b.sc_dev : b.sc;
    if (c.n == (int)kQ8Pad && fast_ratio(sc.adamw))
        step_chunk<PBF16, GBF16, true, true, KEEP, RUNS>(b, sc, c);
    else
        step_chunk<PBF16, GBF16, false, false, KEEP, RUNS>(b, sc, c);
}

template <bool BF16>
__global__ __launch_bounds__(kWave) void q8_encode_kernel(const Q8Batch b) {
    using T = typename GradType<BF16>::T;
    const Chunk c = chunk_of(b, false);
    const int n = c.n, i = threadIdx.x * 4;
    const T* const from_m = c.at<const T>(0);
    const T* const from_v = c.at<const T>(1);
    float m[kBlocks][4] = {}, v[kBlocks][4] = {};
    if (n == (int)kQ8Pad && (c.has & kQ8Has0) && (c.has & kQ8Has1)) {   // no branch between the loads
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            load4<false>(from_m, i + k * (int)kQ8Block, n, true, m[k]);
            load4<false>(from_v, i + k * (int)kQ8Block, n, true, v[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            if (c.has & kQ8Has0) load4<false>(from_m, i + k * (int)kQ8Block, n, false, m[k]);
            if (c.has & kQ8Has1) load4<false>(from_v, i + k * (int)kQ8Block, n, false, v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[k][j] = __uint_as_float(magnitude(v[k][j]));
    store_moments(c, b.sc.key, m, v);
}

template <bool BF16>
__global__ __launch_bounds__(kWave) void q8_decode_kernel(const Q8Batch b) {
    using T = typename GradType<BF16>::T;
    const Chunk c = chunk_of(b, b.runs != 0);
    const int n = c.n;
    const bool whole = n == (int)kQ8Pad;
    uint32_t mc[kBlocks], vc[kBlocks];
    load_codes(c.codes, mc);
    load_codes(c.codes + kQ8Pad, vc);
    const uint32_t scales = uniform(load_scales(c.scales));
    T* const m = c.at<T>(0);
    T* const v = c.at<T>(1);
    wait_loads();
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int i = threadIdx.x * 4 + k * (int)kQ8Block;
        float x[4];
        if (c.has & kQ8Has0) {
            q8_decode4<kTopM>(mc[k], scale_m(scales, k), x);
            store4(m, i, n, whole, x);
        }
        if (c.has & kQ8Has1) {
            q8_decode4<kTopV>(vc[k], scale_v(scales, k), x);
            store4(v, i, n, whole, x);
        }
    }
}

template <bool PBF16, bool GBF16, bool KEEP, bool RUNS>
hipError_t launch_step(const Q8Batch& b, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    const unsigned lds = cap(kStepLds<PBF16, RUNS>, tiles * kQ8Pad);
    if (b.sc_dev != nullptr)
        hipLaunchKernelGGL((adamw_q8_kernel<PBF16, GBF16, true, KEEP, RUNS>), grid, block, lds, stream, b);
    else
        hipLaunchKernelGGL((adamw_q8_kernel<PBF16, GBF16, false, KEEP, RUNS>), grid, block, lds, stream, b);
    return hipGetLastError();
}
template <bool PBF16, bool GBF16>
hipError_t launch_step(const Q8Batch& b, bool keep, int64_t tiles, hipStream_t stream) {
    if (keep)
        return b.runs ? launch_step<PBF16, GBF16, true, true>(b, tiles, stream)
                      : launch_step<PBF16, GBF16, true, false>(b, tiles, stream);
    return b.runs ? launch_step<PBF16, GBF16, false, true>(b, tiles, stream)
                  : launch_step<PBF16, GBF16, false, false>(b, tiles, stream);
}

}  // namespace

hipError_t launch_adamw_q8(const Q8Batch& b, int param_bf16, int grad_bf16, bool keep, int64_t tiles,
                           hipStream_t stream) {
    if (param_bf16)
        return grad_bf16 ? launch_step<true, true>(b, keep, tiles, stream)
                         : launch_step<true, false>(b, keep, tiles, stream);
    return grad_bf16 ? launch_step<false, true>(b, keep, tiles, stream)
                     : launch_step<false, false>(b, keep, tiles, stream);
}

hipError_t launch_q8_encode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    const unsigned lds = cap(bf16 ? 0 : kEncodeLds, tiles * kQ8Pad);
    if (bf16) hipLaunchKernelGGL(q8_encode_kernel<true>, grid, block, lds, stream, b);
    else hipLaunchKernelGGL(q8_encode_kernel<false>, grid, block, lds, stream, b);
    return hipGetLastError();
}

hipError_t launch_q8_decode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    const unsigned lds = cap(b.runs ? kDecodeRunsLds : kDecodeLds, tiles * kQ8Pad);
    if (bf16) hipLaunchKernelGGL(q8_decode_kernel<true>, grid, block, lds, stream, b);
    else hipLaunchKernelGGL(q8_decode_kernel<false>, grid, block, lds, stream, b);
    return hipGetLastError();
}

}  // namespace zs
