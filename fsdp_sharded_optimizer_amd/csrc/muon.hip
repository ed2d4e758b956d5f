// What the matrices' steps do element by element: the new momentum with the
// squares of u, each matrix's inverse norm, u into the products' form, and copies of the
// caller's operands into it.  All HBM-bound.
#include "adamw_math.h"
#include "matrices.h"
#include "reduce.h"

namespace zs {
namespace {

// The clip coefficient as clip_coef forms it; false: no step.
__device__ __forceinline__ bool muon_coef(const MuonScalars& s, const double* norm_sq, float& coef) {
    AdamwScalars a;
    a.clip = s.clip;
    a.max_norm = s.max_norm;
    a.extra_norm_sq = s.extra_norm_sq;
    return clip_coef(a, norm_sq, coef);
}
__device__ __forceinline__ float scaled_grad(const MuonScalars& s, float coef, float g) {
    g = g * s.grad_scale;
    return g * coef;
}
__device__ __forceinline__ float blend(const MuonScalars& s, float m, float g) {
    const float keep = s.momentum * m, add = s.one_minus_momentum * g;
    return keep + add;
}

// m <- momentum m + (1 - momentum) g, and a tile's sum of u^2 (binary64, fixed order).
// Without MOMENTUM: the sum of the input's squares alone.
template <bool GBF16, bool MOMENTUM>
__global__ __launch_bounds__(kBlock) void momentum_kernel(const MomentumBatch b) {
    using G = typename GradType<GBF16>::T;
    uint32_t first;
    const MomentumEntry e = b.e[find_tensor(b.tab, blockIdx.x, first)];
    const G* const grad = unpack_ptr<const G>(e.lo[0], e.hi);
    float* const mom = unpack_ptr<float>(e.lo[1], e.hi >> 16);
    const MuonScalars& sc = b.sc_dev ? *b.sc_dev : b.sc;
    const int64_t at0 = (int64_t)(blockIdx.x - first) * kMomentumTile + threadIdx.x * 4, n = e.numel;
    constexpr int kQ = (int)(kMomentumTile / (kBlock * 4));
    double s0 = 0.0, s1 = 0.0;
    float coef = 1.0f;
    if (at0 - threadIdx.x * 4 + kMomentumTile <= n) {
        f32x4 g[kQ], m[kQ];
#pragma unroll
        for (int q = 0; q < kQ; ++q) g[q] = ld4<true>(grad + at0 + q * kBlock * 4);
        if constexpr (MOMENTUM) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) m[q] = ld4<true>(mom + at0 + q * kBlock * 4);
            if (!muon_coef(sc, b.norm_sq, coef)) return;
        }
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            float u[4] = {g[q].x, g[q].y, g[q].z, g[q].w};
            if constexpr (MOMENTUM) {
                float v[4] = {m[q].x, m[q].y, m[q].z, m[q].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float gj = scaled_grad(sc, coef, u[j]);
                    v[j] = blend(sc, v[j], gj);
                    u[j] = sc.nesterov ? blend(sc, v[j], gj) : v[j];
                }
                *reinterpret_cast<f32x4_any*>(mom + at0 + q * kBlock * 4) = f32x4{v[0], v[1], v[2], v[3]};
            }
            add_squares4(u, 1.0f, s0, s1);
        }
    } else {
        if (MOMENTUM && !muon_coef(sc, b.norm_sq, coef)) return;
#pragma unroll 1
        for (int q = 0; q < kQ; ++q)
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const int64_t i = at0 + q * kBlock * 4 + j;
                if (i >= n) continue;
                float u = widen(grad[i]);
                if constexpr (MOMENTUM) {
                    const float gj = scaled_grad(sc, coef, u), v = blend(sc, mom[i], gj);
                    mom[i] = v;
                    u = sc.nesterov ? blend(sc, v, gj) : v;
                }
                s0 = __builtin_fma((double)u, (double)u, s0);
            }
    }
    const double total = block_sum(s0 + s1);
    if (threadIdx.x == 0) b.partials[blockIdx.x] = total;
}

// kNsScale over a matrix's norm; a norm that is not finite makes all of it NaN
__device__ __forceinline__ float inverse_norm(double squares, double eps) {
    const double norm = sqrt(squares);
    return __builtin_isfinite(norm) ? (float)((double)kNsScale / (norm > eps ? norm : eps)) : __builtin_nanf("");
}

__global__ __launch_bounds__(kBlock) void inverse_norms_kernel(const NormsBatch b) {
    const uint32_t from = b.start[blockIdx.x], to = b.start[blockIdx.x + 1];
    double s = 0.0;
    for (uint32_t i = from + threadIdx.x; i < to; i += kBlock) s += b.partials[i];
    s = block_sum(s);
    if (threadIdx.x == 0) b.inverse[blockIdx.x] = inverse_norm(s, b.sc_dev ? b.sc_dev->eps : b.eps);
}

// eight consecutive elements of a row, zeros past its end
template <typename G>
__device__ __forceinline__ void load8(const G* row, int64_t c, int64_t cols, float (&x)[8]) {
    if (c + 8 <= cols) {
        const f32x4 a = ld4<true>(row + c), b = ld4<true>(row + c + 4);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = v[j];
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? widen(row[c + j]) : 0.0f;
}

constexpr int kSide = (int)kPadSide;

// A 64 x 64 tile of a matrix (value(row, column, x): eight values of a row of the
// source), given to store(row, column, x) by rows of the destination; TALL: the
// destination is the source's transpose.
template <class Value, class Store>
__device__ __forceinline__ void move_tile(bool transposed, int64_t r0, int64_t c0, Value&& value, Store&& store) {
    __shared__ float t[kSide][kSide + 1];
    const int c = (threadIdx.x % 8) * 8, r = threadIdx.x / 8;
    float x[8];
    if (!transposed) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            value(r0 + r + 32 * h, c0 + c, x);
            store(r0 + r + 32 * h, c0 + c, x);
        }
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        value(c0 + r + 32 * h, r0 + c, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[r + 32 * h][c + j] = x[j];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = t[c + j][r + 32 * h];
        store(r0 + r + 32 * h, c0 + c, x);
    }
}

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <bool GBF16, bool MOMENTUM>
__global__ __launch_bounds__(kBlock) void pack_kernel(const PackBatch b) {
    using G = typename GradType<GBF16>::T;
    uint32_t first;
    const uint32_t k = find_tensor(b.tab, blockIdx.x, first);
    const PackEntry e = b.e[k];
    const G* const grad = unpack_ptr<const G>(e.lo[0], e.hi);
    const float* const mom = unpack_ptr<const float>(e.lo[1], e.hi >> 16);
    const MuonScalars& sc = b.sc_dev ? *b.sc_dev : b.sc;
    float coef = 1.0f;
    if (MOMENTUM && !muon_coef(sc, b.norm_sq, coef)) return;
    const bool tall = (e.n & kTall) != 0;
    const int64_t m = e.m, n = e.n & ~kTall, rows = tall ? n : m, cols = tall ? m : n;
    const NsPlace p(m, n);
    const uint32_t across = (uint32_t)(p.np / kSide), tile = blockIdx.x - first;
    float scale;
    if (b.inverse != nullptr) {
        scale = b.inverse[k];
    } else {
        __shared__ float formed;
        const int64_t count = (m * n + kMomentumTile - 1) / kMomentumTile;
        const double s = block_sum(threadIdx.x < count ? b.partials[e.partial + threadIdx.x] : 0.0);
        if (threadIdx.x == 0) formed = inverse_norm(s, sc.eps);
        __syncthreads();
        scale = formed;
    }
    char* const base = b.ws + (int64_t)e.base * kNsUnit;
    _Float16* const hi = reinterpret_cast<_Float16*>(base + p.hi(0));
    _Float16* const lo = reinterpret_cast<_Float16*>(base + p.lo(0));
    // a skinny matrix's first values again, behind the second ones
    _Float16* const again = m <= kSkinny ? reinterpret_cast<_Float16*>(base + 2 * p.x) : nullptr;
    move_tile(tall, (int64_t)(tile / across) * kSide, (int64_t)(tile % across) * kSide,
        [&](int64_t r, int64_t c, float (&x)[8]) {
            if (r >= rows) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.0f;
                return;
            }
            if (!MOMENTUM || sc.nesterov) load8(grad + r * cols, c, cols, x);
            if constexpr (MOMENTUM) {
                float v[8];
                load8(mom + r * cols, c, cols, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = sc.nesterov ? blend(sc, v[j], scaled_grad(sc, coef, x[j])) : v[j];
            }
        },
        [&](int64_t r, int64_t c, const float (&x)[8]) {
            f16x8 h, l;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                _Float16 first_of, second_of;
                split_f16(x[j] * scale, first_of, second_of);
                h[j] = first_of;
                l[j] = second_of;
            }
            // (a tile is a block of the workspace)
            const int64_t at = (int64_t)tile * (kSide * kSide) + (r % kSide) * kSide + c % kSide;
            *reinterpret_cast<f16x8*>(hi + at) = h;
            *reinterpret_cast<f16x8*>(lo + at) = l;
            if (again != nullptr) *reinterpret_cast<f16x8*>(again + at) = h;
        });
}

// x as two bf16 values; the first towards zero where to nearest would be infinite
__device__ __forceinline__ void split_bf16(float x, uint32_t& hi, uint32_t& lo) {
    hi = f32_to_bf16_rne(x);
    if ((hi & 0x7FFFu) == 0x7F80u) hi = __float_as_uint(x) >> 16;
    lo = f32_to_bf16_rne(x - bf16_to_f32(hi));
}

template <bool SBF16, int KIND>
__global__ __launch_bounds__(kBlock) void stage_kernel(const StageBatch b, int k_rows, int transposed) {
    using S = typename GradType<SBF16>::T;
    uint32_t first;
    const StageEntry e = b.e[find_tensor(b.tab, blockIdx.x, first)];
    const S* const src = unpack_ptr<const S>(e.lo[0], e.hi);
    uint16_t* const dst = unpack_ptr<uint16_t>(e.lo[1], e.hi >> 16);
    const int64_t rows = e.rows, cols = e.cols, pr = pad_side(rows), pc = pad_side(cols);
    const int64_t src_rows = transposed ? cols : rows, src_cols = transposed ? rows : cols;
    const uint32_t across = (uint32_t)(pc / kSide), tile = blockIdx.x - first;
    constexpr int kParts = KIND == kStagePlain ? 1 : 3;
    const int64_t pitch = k_rows ? pc : pc * kParts, part = k_rows ? pr * pc : pc;
    move_tile(transposed != 0, (int64_t)(tile / across) * kSide, (int64_t)(tile % across) * kSide,
        [&](int64_t r, int64_t c, float (&x)[8]) {
            if (r < src_rows) {
                load8(src + r * src_cols, c, src_cols, x);
                return;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
        },
        [&](int64_t r, int64_t c, const float (&x)[8]) {
            u32x4 h = {0, 0, 0, 0}, l = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t hj, lj = 0;
                if constexpr (KIND == kStagePlain) hj = f32_to_bf16_rne(x[j]);
                else split_bf16(x[j], hj, lj);
                h[j / 2] |= hj << (16 * (j % 2));
                l[j / 2] |= lj << (16 * (j % 2));
            }
            uint16_t* const to = dst + r * pitch + c;
            *reinterpret_cast<u32x4*>(to) = h;
            if constexpr (KIND == kStageHiHiLo) {
                *reinterpret_cast<u32x4*>(to + part) = h;
                *reinterpret_cast<u32x4*>(to + 2 * part) = l;
            } else if constexpr (KIND == kStageHiLoHi) {
                *reinterpret_cast<u32x4*>(to + part) = l;
                *reinterpret_cast<u32x4*>(to + 2 * part) = h;
            }
        });
}

}  // namespace

hipError_t launch_momentum(const MomentumBatch& b, int grad_bf16, bool momentum, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kBlock);
    if (grad_bf16 && momentum) hipLaunchKernelGGL((momentum_kernel<true, true>), grid, block, 0, stream, b);
    else if (grad_bf16) hipLaunchKernelGGL((momentum_kernel<true, false>), grid, block, 0, stream, b);
    else if (momentum) hipLaunchKernelGGL((momentum_kernel<false, true>), grid, block, 0, stream, b);
    else hipLaunchKernelGGL((momentum_kernel<false, false>), grid, block, 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_inverse_norms(const NormsBatch& b, hipStream_t stream) {
    hipLaunchKernelGGL(inverse_norms_kernel, dim3(b.count), dim3(kBlock), 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_pack(const PackBatch& b, int grad_bf16, bool momentum, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kBlock);
    if (grad_bf16 && momentum) hipLaunchKernelGGL((pack_kernel<true, true>), grid, block, 0, stream, b);
    else if (grad_bf16) hipLaunchKernelGGL((pack_kernel<true, false>), grid, block, 0, stream, b);
    else if (momentum) hipLaunchKernelGGL((pack_kernel<false, true>), grid, block, 0, stream, b);
    else hipLaunchKernelGGL((pack_kernel<false, false>), grid, block, 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_stage(const StageBatch& b, int src_bf16, int kind, bool k_rows, bool transposed, int64_t tiles,
                        hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kBlock);
    const int kr = k_rows, tr = transposed;
    if (src_bf16) hipLaunchKernelGGL((stage_kernel<true, kStagePlain>), grid, block, 0, stream, b, kr, tr);
    else if (kind == kStageHiHiLo) hipLaunchKernelGGL((stage_kernel<false, kStageHiHiLo>), grid, block, 0, stream, b, kr, tr);
    else hipLaunchKernelGGL((stage_kernel<false, kStageHiLoHi>), grid, block, 0, stream, b, kr, tr);
    return hipGetLastError();
}

}  // namespace zs
