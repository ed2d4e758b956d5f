// AdamW over a list of tensors with 8-bit moments, and the conversions of
// such moments.
//
// The step decodes a block's moments, forms the new ones as the fp32 step does
// (the operations and roundings of adamw_math.h: codes hang on their last
// bits), updates the parameter, takes the block's two new scales from the
// largest magnitudes and stores the codes: 4 bytes of moments per element
// (read and written) instead of 16.
//
// A wave takes one chunk of kQ8Pad = 1024 elements, 4 blocks, 16 elements per
// lane: what a wave does once (finding its tensor, the clip coefficient in
// binary64, one access for all its codes) is then spread over 16 elements.
#include "adamw_math.h"
#include "q8.h"

namespace zs {
namespace {

constexpr int kWave = 64;
constexpr int kBlocks = (int)(kQ8Pad / kQ8Block);   // per wave
// LDS reserved (never touched) per workgroup to cap how many share a CU: too
// many keep too many DRAM rows open.  Measured on 809M fp32 parameters with bf16
// gradients and re-casts (855M bf16 parameters; 317M moments to and from bf16),
// of the 8 TB/s peak: step 73.1 % at 6 KiB, 75.5 at 8, 76.4 at 10, 77.3 at 12,
// 77.6 at 14, 76.4 at 16 (bf16: 78.7 at 6, 79.6 at 8, 79.8 at 10, 78.6 at 12, 74.7 at
// 14: fewer bytes per wave want more waves); read-out 75.9 % uncapped, 78.9 at
// 8 KiB, 68.2 at 12; storing 68.1 % uncapped, 70.3 at 4 KiB, 60.4 at 6.  Two blocks
// per wave instead of four: the step within 0.3 points at its best cap, storing
// 4 points slower; 2 or 4 waves per workgroup: 0.5-4 points slower; plain instead
// of streaming code accesses: the step 1 point slower.  A launch of fewer than
// 32768 chunks (34M elements) is not long enough for that and ends sooner with
// more of it resident: 8.4M bf16 parameters 19.6 us uncapped, 21.2 at 10 KiB; 34M
// 59.0 and 61.0; read out 10.4 and 10.9 at 8 KiB.
template <bool PBF16> constexpr unsigned kStepLds = PBF16 ? 10240 : 14336;
constexpr unsigned kEncodeLds = 4096;
constexpr unsigned kDecodeLds = 8192;
constexpr int64_t kCapChunks = 32768;
unsigned cap(unsigned lds, int64_t chunks) { return chunks < kCapChunks ? 0 : lds; }

// Where a wave works: its tensor's entry and its chunk.
struct Chunk {
    Q8Entry e;
    int64_t first;     // of the entry, of the chunk's elements
    int64_t i;         // of the lane's first block's elements
    uint8_t* m;        // the lane's codes
    uint8_t* v;
    uint2* scales;     // the chunk's
};
__device__ __forceinline__ Chunk chunk_of(const Q8Batch& b) {
    uint32_t first_tile;
    const Q8Entry e = b.e[find_tensor(b.tab, blockIdx.x, first_tile)];
    const Q8At at = q8_at(e);
    const int64_t first = (int64_t)(blockIdx.x - first_tile) * kQ8Pad;
    return Chunk{e, first, first + threadIdx.x * 4,
                 at.codes + 2 * first + threadIdx.x * 16, at.codes + 2 * first + kQ8Pad + threadIdx.x * 16,
                 reinterpret_cast<uint2*>(at.scales + first / (kQ8Block / 2))};
}

// 4 consecutive elements from i of n (zeros past the end).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int64_t i, int64_t n, bool whole, float (&x)[4]) {
    if (whole || i + 4 <= n) {
        const f32x4 w = ld4(p + i);
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
__device__ __forceinline__ void store4(T* p, int64_t i, int64_t n, bool whole, const float (&x)[4]) {
    if (whole || i + 4 <= n) {
        st4_hw(p + i, f32x4{x[0], x[1], x[2], x[3]});
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) st1(p + i + j, x[j]);
    }
}
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[kBlocks]) {
    const u32x4 x = ld_stream(reinterpret_cast<const u32x4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[kBlocks]) {
    st_stream(reinterpret_cast<u32x4*>(p), u32x4{w[0], w[1], w[2], w[3]});
}

// The chunk's scale bytes as two words: block b's exp_avg byte and exp_avg_sq
// byte are the bytes 2b and 2b + 1.
__device__ __forceinline__ uint32_t scale_m(const uint2& s, int b) {
    return ((b < 2 ? s.x : s.y) >> (16 * (b & 1))) & 0xFFu;
}
__device__ __forceinline__ uint32_t scale_v(const uint2& s, int b) {
    return ((b < 2 ? s.x : s.y) >> (16 * (b & 1) + 8)) & 0xFFu;
}

// Stores the moments of a chunk: the blocks' scales from their largest
// magnitudes, then the codes.
__device__ __forceinline__ void store_moments(const Chunk& c, uint32_t key, const float (&m)[kBlocks][4],
                                              const float (&v)[kBlocks][4]) {
    static_assert(kBlocks == 4, "8 maxima");
    uint32_t most[2 * kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) most[2 * b] = max4(m[b]), most[2 * b + 1] = max4(v[b]);
    const uint32_t e = q8_scale(wave_max8(most));
    uint32_t mc[kBlocks], vc[kBlocks];
    uint32_t scales[2] = {0, 0};
    const uint32_t tensor_key = q8_mix(key + (c.e.index_off & 0xFFFFFFu) * kGolden);
    // the chunk's first group; its 256 groups share the upper 32 bits
    const uint32_t group = q8_group(((uint64_t)(c.e.index_off >> 24) * kLaunchElems + (uint64_t)c.first) / 4, tensor_key);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const uint32_t em = (uint32_t)__builtin_amdgcn_readlane((int)e, max8_lane(2 * b));
        const uint32_t ev = (uint32_t)__builtin_amdgcn_readlane((int)e, max8_lane(2 * b + 1));
        const uint32_t word = q8_mix(group + b * (uint32_t)(kQ8Block / 4) + threadIdx.x);
        mc[b] = q8_encode4<kTopM>(m[b], em, word);
        vc[b] = q8_encode4<kTopV>(v[b], ev, word);
        scales[b / 2] |= (em | ev << 8) << (16 * (b & 1));
    }
    store_codes(c.m, mc);
    store_codes(c.v, vc);
    if (threadIdx.x == 0) *c.scales = uint2{scales[0], scales[1]};
}

// u / step_size of one element from its new moments
template <bool FAST>
__device__ __forceinline__ float adam_ratio(const AdamwScalars& a, float inv_root, float m, float v) {
    if constexpr (FAST) {
        // The hardware's square root and reciprocal are within 1 ulp: u is
        // within 8 * 2^-24 of the exact quotient, far below the parameter's
        // own rounding, for 11 issue slots against about 50 for IEEE division
        // and root.  They flush subnormals: den is at least eps, and a
        // subnormal v's root is below 2^-63.
        const float den = __builtin_fmaf(__builtin_amdgcn_sqrtf(v), inv_root, a.eps);
        return m * __builtin_amdgcn_rcpf(den);
    }
    float den = sqrtf(v) / a.bias_correction2_sqrt;
    den = den + a.eps;
    return m / den;
}
constexpr float kFastEps = 0x1p-40f;

// One chunk's step.  WHOLE: all its elements are the tensor's.
template <bool PBF16, bool GBF16, bool WHOLE, bool FAST>
__device__ __forceinline__ void step_chunk(const Q8Batch& b, const Q8Scalars& sc, const Chunk& c) {
    using P = typename GradType<PBF16>::T;
    using G = typename GradType<GBF16>::T;
    const int64_t n = c.e.numel;
    P* const param = unpack_ptr<P>(c.e.lo[0], c.e.hi[0]);
    const G* const grad = unpack_ptr<const G>(c.e.lo[1], c.e.hi[0] >> 16);
    uint16_t* const copy = unpack_ptr<uint16_t>(c.e.lo[3], c.e.hi[1] >> 16);
    float g[kBlocks][4], p[kBlocks][4], m[kBlocks][4], v[kBlocks][4];
    uint32_t mc[kBlocks], vc[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) load4(grad, c.i + k * kQ8Block, n, WHOLE, g[k]);
    load_codes(c.m, mc);
    load_codes(c.v, vc);
    uint2 scales = *c.scales;
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) load4(param, c.i + k * kQ8Block, n, WHOLE, p[k]);
    float coef;
    if (!clip_coef(sc.adamw, b.norm_sq, coef)) return;
    scales.x = (uint32_t)__builtin_amdgcn_readfirstlane((int)scales.x);
    scales.y = (uint32_t)__builtin_amdgcn_readfirstlane((int)scales.y);
    const AdamwScalars& a = sc.adamw;
    const float inv_root = 1.0f / a.bias_correction2_sqrt;
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const uint32_t em = scale_m(scales, k), ev = scale_v(scales, k);
        // beta * value: the scale, a power of two, goes into the factor, which
        // changes no bit of the product
        float keep_m = a.beta1, keep_v = a.beta2;
        if (plain_scale<kTopM>(em) && plain_scale<kTopV>(ev)) {
            q8_unpack4<kTopM>(mc[k], m[k]);
            q8_unpack4<kTopV>(vc[k], v[k]);
            keep_m *= exp2_of((int)em - kTopM);
            keep_v *= exp2_of((int)ev - kTopV);
        } else {
            q8_decode4<kTopM>(mc[k], em, m[k]);
            q8_decode4<kTopV>(vc[k], ev, v[k]);
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
            if (!WHOLE && c.i + k * kQ8Block + j >= n) m[k][j] = v[k][j] = 0.0f;
        }
        store4(param, c.i + k * kQ8Block, n, WHOLE, p[k]);
        if (!PBF16 && copy != nullptr) store4(copy, c.i + k * kQ8Block, n, WHOLE, p[k]);
    }
    store_moments(c, sc.key, m, v);
}

template <bool PBF16, bool GBF16, bool DEV>
__global__ __launch_bounds__(kWave) void adamw_q8_kernel(const Q8Batch b) {
    const Chunk c = chunk_of(b);
    const Q8Scalars sc = DEV ? *b.sc_dev : b.sc;
    if (c.first + kQ8Pad <= (int64_t)c.e.numel && sc.adamw.eps >= kFastEps) step_chunk<PBF16, GBF16, true, true>(b, sc, c);
    else step_chunk<PBF16, GBF16, false, false>(b, sc, c);
}

template <bool BF16>
__global__ __launch_bounds__(kWave) void q8_encode_kernel(const Q8Batch b) {
    using T = typename GradType<BF16>::T;
    const Chunk c = chunk_of(b);
    const int64_t n = c.e.numel;
    const bool whole = c.first + kQ8Pad <= n;
    const T* const from_m = unpack_ptr<const T>(c.e.lo[0], c.e.hi[0]);
    const T* const from_v = unpack_ptr<const T>(c.e.lo[1], c.e.hi[0] >> 16);
    float m[kBlocks][4] = {}, v[kBlocks][4] = {};
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int64_t i = c.i + k * kQ8Block;
        if (from_m != nullptr) load4(from_m, i, n, whole, m[k]);
        if (from_v != nullptr) load4(from_v, i, n, whole, v[k]);
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
    const Chunk c = chunk_of(b);
    const int64_t n = c.e.numel;
    const bool whole = c.first + kQ8Pad <= n;
    uint32_t mc[kBlocks], vc[kBlocks];
    load_codes(c.m, mc);
    load_codes(c.v, vc);
    uint2 scales = *c.scales;
    scales.x = (uint32_t)__builtin_amdgcn_readfirstlane((int)scales.x);
    scales.y = (uint32_t)__builtin_amdgcn_readfirstlane((int)scales.y);
    T* const m = unpack_ptr<T>(c.e.lo[0], c.e.hi[0]);
    T* const v = unpack_ptr<T>(c.e.lo[1], c.e.hi[0] >> 16);
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int64_t i = c.i + k * kQ8Block;
        float x[4];
        if (m != nullptr) {
            q8_decode4<kTopM>(mc[k], scale_m(scales, k), x);
            store4(m, i, n, whole, x);
        }
        if (v != nullptr) {
            q8_decode4<kTopV>(vc[k], scale_v(scales, k), x);
            store4(v, i, n, whole, x);
        }
    }
}

template <bool PBF16, bool GBF16>
hipError_t launch_step(const Q8Batch& b, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    if (b.sc_dev != nullptr)
        hipLaunchKernelGGL((adamw_q8_kernel<PBF16, GBF16, true>), grid, block, cap(kStepLds<PBF16>, tiles), stream, b);
    else
        hipLaunchKernelGGL((adamw_q8_kernel<PBF16, GBF16, false>), grid, block, cap(kStepLds<PBF16>, tiles), stream, b);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw_q8(const Q8Batch& b, int param_bf16, int grad_bf16, int64_t tiles, hipStream_t stream) {
    if (param_bf16)
        return grad_bf16 ? launch_step<true, true>(b, tiles, stream) : launch_step<true, false>(b, tiles, stream);
    return grad_bf16 ? launch_step<false, true>(b, tiles, stream) : launch_step<false, false>(b, tiles, stream);
}

hipError_t launch_q8_encode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    if (bf16) hipLaunchKernelGGL(q8_encode_kernel<true>, grid, block, cap(kEncodeLds, tiles), stream, b);
    else hipLaunchKernelGGL(q8_encode_kernel<false>, grid, block, cap(kEncodeLds, tiles), stream, b);
    return hipGetLastError();
}

hipError_t launch_q8_decode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    if (bf16) hipLaunchKernelGGL(q8_decode_kernel<true>, grid, block, cap(kDecodeLds, tiles), stream, b);
    else hipLaunchKernelGGL(q8_decode_kernel<false>, grid, block, cap(kDecodeLds, tiles), stream, b);
    return hipGetLastError();
}

}  // namespace zs
