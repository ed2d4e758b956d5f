// AdamW over a list of tensors with 8-bit moments, and the conversions of
// such moments.
//
// The step decodes a block's moments, forms the new ones and the parameter as
// the fp32 step does (adamw_math.h), takes the block's two new scales from the
// largest magnitudes and stores the codes: 4 bytes of moments per element
// (read and written) instead of 16.
#include "adamw_math.h"
#include "q8.h"

namespace zs {
namespace {

constexpr int kWave = 64;

// Up to 4 consecutive elements from `i` of n (zeros past the end).
template <typename T>
__device__ __forceinline__ void load_upto4(const T* p, int64_t i, int64_t n, float (&x)[4]) {
    if (i + 4 <= n) {
        const f32x4 w = ld4(p + i);
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = i + j < n ? widen(p[i + j]) : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store_upto4(T* p, int64_t i, int64_t n, const float (&x)[4]) {
    if (i + 4 <= n) {
        st4(p + i, f32x4{x[0], x[1], x[2], x[3]});
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) st1(p + i + j, x[j]);
    }
}
// the code word of 4 elements from i (a multiple of 4: inside the padded codes)
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int64_t n) {
    return i < n ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p + i)) : 0u;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, uint32_t w) {
    if (i < n) __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(p + i));
}
// both scale bytes of the block that starts at element i (uniform)
__device__ __forceinline__ uint16_t* scale_at(const Q8At& at, int64_t i) {
    return reinterpret_cast<uint16_t*>(at.scales + i / (kQ8Block / 2));
}

template <bool PBF16, bool GBF16, bool DEV>
__global__ __launch_bounds__(kWave) void adamw_q8_kernel(const Q8Batch b) {
    using P = typename GradType<PBF16>::T;
    using G = typename GradType<GBF16>::T;
    uint32_t first;
    const int t = find_tensor(b.tab, blockIdx.x, first);
    const Q8Entry& e = b.e[t];
    const Q8Scalars sc = DEV ? *b.sc_dev : b.sc;
    const Q8At at = q8_at(e);
    const int64_t n = e.numel;
    const int64_t block = (int64_t)(blockIdx.x - first) * kQ8Block;
    const int64_t i = block + threadIdx.x * 4;
    float g[4], p[4], m[4], v[4];
    load_upto4(static_cast<const G*>(e.grad), i, n, g);
    load_upto4(static_cast<const P*>(e.param), i, n, p);
    const uint32_t mc = load_codes(at.m, i, n), vc = load_codes(at.v, i, n);
    const uint32_t scales = (uint32_t)__builtin_amdgcn_readfirstlane(*scale_at(at, block));
    float coef;
    if (!clip_coef(sc.adamw, b.norm_sq, coef)) return;
    q8_decode4<kTopM>(mc, scales & 0xFFu, m);
    q8_decode4<kTopV>(vc, scales >> 8, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float u = adam_elem(sc.adamw, coef, g[j], m[j], v[j]);
        p[j] = apply_step(sc.adamw, p[j], u);
        if (i + j >= n) m[j] = v[j] = 0.0f;   // past the end: no part of the block's scale
    }
    store_upto4(static_cast<P*>(e.param), i, n, p);
    if (!PBF16 && e.copy != nullptr) store_upto4(static_cast<uint16_t*>(e.copy), i, n, p);
    const uint32_t em = q8_scale(wave_max(max4(m))), ev = q8_scale(wave_max(max4(v)));
    const uint64_t group = ((uint64_t)e.off * kQ8Pad + (uint64_t)i) / 4;
    const uint32_t word = q8_word(group, q8_mix(sc.key + e.index * kGolden));
    store_codes(at.m, i, n, q8_encode4<kTopM>(m, em, word));
    store_codes(at.v, i, n, q8_encode4<kTopV>(v, ev, word));
    if (threadIdx.x == 0) *scale_at(at, block) = (uint16_t)(em | ev << 8);
}

template <bool BF16>
__global__ __launch_bounds__(kWave) void q8_encode_kernel(const Q8Batch b) {
    using T = typename GradType<BF16>::T;
    uint32_t first;
    const int t = find_tensor(b.tab, blockIdx.x, first);
    const Q8Entry& e = b.e[t];
    const Q8At at = q8_at(e);
    const int64_t n = e.numel;
    const int64_t block = (int64_t)(blockIdx.x - first) * kQ8Block;
    const int64_t i = block + threadIdx.x * 4;
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f}, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (e.param != nullptr) load_upto4(static_cast<const T*>(e.param), i, n, m);
    if (e.grad != nullptr) load_upto4(static_cast<const T*>(e.grad), i, n, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(magnitude(v[j]));
    const uint32_t em = q8_scale(wave_max(max4(m))), ev = q8_scale(wave_max(max4(v)));
    const uint64_t group = ((uint64_t)e.off * kQ8Pad + (uint64_t)i) / 4;
    const uint32_t word = q8_word(group, q8_mix(b.sc.key + e.index * kGolden));
    store_codes(at.m, i, n, q8_encode4<kTopM>(m, em, word));
    store_codes(at.v, i, n, q8_encode4<kTopV>(v, ev, word));
    if (threadIdx.x == 0) *scale_at(at, block) = (uint16_t)(em | ev << 8);
}

template <bool BF16>
__global__ __launch_bounds__(kWave) void q8_decode_kernel(const Q8Batch b) {
    using T = typename GradType<BF16>::T;
    uint32_t first;
    const int t = find_tensor(b.tab, blockIdx.x, first);
    const Q8Entry& e = b.e[t];
    const Q8At at = q8_at(e);
    const int64_t n = e.numel;
    const int64_t block = (int64_t)(blockIdx.x - first) * kQ8Block;
    const int64_t i = block + threadIdx.x * 4;
    const uint32_t mc = load_codes(at.m, i, n), vc = load_codes(at.v, i, n);
    const uint32_t scales = (uint32_t)__builtin_amdgcn_readfirstlane(*scale_at(at, block));
    float x[4];
    if (e.param != nullptr) {
        q8_decode4<kTopM>(mc, scales & 0xFFu, x);
        store_upto4(static_cast<T*>(e.param), i, n, x);
    }
    if (e.copy != nullptr) {
        q8_decode4<kTopV>(vc, scales >> 8, x);
        store_upto4(static_cast<T*>(e.copy), i, n, x);
    }
}

template <bool PBF16, bool GBF16>
hipError_t launch_step(const Q8Batch& b, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    if (b.sc_dev != nullptr)
        hipLaunchKernelGGL((adamw_q8_kernel<PBF16, GBF16, true>), grid, block, 0, stream, b);
    else
        hipLaunchKernelGGL((adamw_q8_kernel<PBF16, GBF16, false>), grid, block, 0, stream, b);
    return hipGetLastError();
}

}  // namespace

int64_t q8_step_tile() { return kQ8Block; }
int64_t q8_codec_tile() { return kQ8Block; }

hipError_t launch_adamw_q8(const Q8Batch& b, int param_bf16, int grad_bf16, int64_t tiles, hipStream_t stream) {
    if (param_bf16)
        return grad_bf16 ? launch_step<true, true>(b, tiles, stream) : launch_step<true, false>(b, tiles, stream);
    return grad_bf16 ? launch_step<false, true>(b, tiles, stream) : launch_step<false, false>(b, tiles, stream);
}

hipError_t launch_q8_encode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    if (bf16) hipLaunchKernelGGL(q8_encode_kernel<true>, grid, block, 0, stream, b);
    else hipLaunchKernelGGL(q8_encode_kernel<false>, grid, block, 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_q8_decode(const Q8Batch& b, int bf16, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kWave);
    if (bf16) hipLaunchKernelGGL(q8_decode_kernel<true>, grid, block, 0, stream, b);
    else hipLaunchKernelGGL(q8_decode_kernel<false>, grid, block, 0, stream, b);
    return hipGetLastError();
}

}  // namespace zs
