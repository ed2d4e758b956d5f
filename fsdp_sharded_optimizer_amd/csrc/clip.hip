// The squared norms of a list of gradients in fp32 and bf16, of each tensor and of
// all, and their clipping.
//
// Norms: a tile's sum of squares as in norm_tensors.hip (norm_tile.h), here with a
// tensor's dtype in its record; then each tensor's partials, then the tensors',
// every sum in binary64 and in an order that only the numels and dtypes fix.
// HBM-bound: each gradient read once.
//
// Clipping: y = fl(fl(widen(g) * scale) * coef), rounded to the destination's dtype.
// HBM-bound: read once, written once.
#include "adamw_math.h"
#include "clip.h"
#include "norm_tile.h"

namespace zs {
namespace {

template <bool KEEP>
__global__ __launch_bounds__(kBlock) void norms_kernel(const NormBatch b, float scale, double* __restrict__ partials) {
    uint32_t first;
    const uint32_t t = find_tensor(b.tab, blockIdx.x, first);
    const NormEntry e = b.e[t];
    const bool last = blockIdx.x + 1 == b.tab.start[t + 1], bf16 = (e.hi_tail & kNormBf16) != 0;
    const int tail = (int)((e.hi_tail >> 16) & 0x7FFFu) + 1;
    const uint16_t* const p = unpack_ptr<const uint16_t>(e.lo, e.hi_tail);
    double s;
    if (bf16) {
        const uint16_t* const g = p + (int64_t)(blockIdx.x - first) * kNormTile<true>;
        s = norm_tile<true, KEEP>(g, last ? tail : (int)kNormTile<true>, last, (e.lo & 2) != 0, scale);
    } else {
        const float* const g = reinterpret_cast<const float*>(p) + (int64_t)(blockIdx.x - first) * kNormTile<false>;
        s = norm_tile<false, KEEP>(g, last ? tail : (int)kNormTile<false>, last, false, scale);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partials[xcd_slot(blockIdx.x, gridDim.x)] = s;
}

__global__ __launch_bounds__(kBlock) void tensor_sums_kernel(const TensorSums b) {
    const uint32_t to = b.start[blockIdx.x + 1];
    double s = 0.0;
    for (uint32_t i = b.start[blockIdx.x] + threadIdx.x; i < to; i += kBlock) s += b.partials[xcd_slot(i, b.grid)];
    s = block_sum(s);
    if (threadIdx.x == 0) b.norms[blockIdx.x] = s;
}

__global__ __launch_bounds__(kBlock) void total_kernel(const double* __restrict__ norms, int64_t count,
                                                       double* __restrict__ out) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kBlock) s += norms[i];
    s = block_sum(s);
    if (threadIdx.x == 0) *out = s;
}

// Both in one workgroup, for a list of few tensors and partials: a wave adds the
// partials of every 16th tensor, the first wave the tensors.
constexpr int kFewThreads = 1024;
__global__ __launch_bounds__(kFewThreads) void few_sums_kernel(const TensorSums b, double* __restrict__ out) {
    __shared__ double norm[kFewTensors];
    const uint32_t lane = threadIdx.x % 64;
    for (uint32_t k = threadIdx.x / 64; k < b.count; k += kFewThreads / 64) {
        const uint32_t to = b.start[k + 1];
        double s = 0.0;
        for (uint32_t i = b.start[k] + lane; i < to; i += 64) s += b.partials[xcd_slot(i, b.grid)];
        s = wave_sum(s);
        if (lane == 0) {
            norm[k] = s;
            b.norms[k] = s;
        }
    }
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const double s = wave_sum(lane < b.count ? norm[lane] : 0.0);
    if (lane == 0) *out = s;
}

template <typename S, typename D>
__device__ __forceinline__ void clip_tile(const S* src, D* dst, int64_t n, int64_t tile, float scale, float coef) {
    constexpr int kQ = (int)(kClipTile / (kBlock * 4));
    const int64_t at = tile * kClipTile + threadIdx.x * 4;
    if ((tile + 1) * kClipTile <= n) {
        f32x4 x[kQ];
#pragma unroll
        for (int q = 0; q < kQ; ++q) x[q] = ld4(src + at + q * kBlock * 4);
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            x[q] = x[q] * scale;
            st4(dst + at + q * kBlock * 4, x[q] * coef);
        }
        return;
    }
#pragma unroll 1
    for (int q = 0; q < kQ; ++q)
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const int64_t i = at + q * kBlock * 4 + j;
            if (i >= n) continue;
            const float g = widen(src[i]) * scale;
            st1(dst + i, g * coef);
        }
}

__global__ __launch_bounds__(kBlock) void clip_kernel(const ClipBatch b) {
    uint32_t first;
    const uint32_t t = find_tensor(b.tab, blockIdx.x, first), bf16 = b.bf16[t / 16] >> (2 * (t % 16)) & 3u;
    const ClipEntry e = b.e[t];
    AdamwScalars sc;
    sc.clip = b.clip;
    sc.max_norm = b.max_norm;
    sc.extra_norm_sq = b.extra_norm_sq;
    float coef;
    if (!clip_coef(sc, b.norm_sq, coef)) return;
    const void* const src = unpack_ptr<const uint16_t>(e.lo[0], e.hi);
    void* const dst = unpack_ptr<uint16_t>(e.lo[1], e.hi >> 16);
    // in place, times one: as it is
    if (src == dst && b.scale == 1.0f && coef == 1.0f) return;
    const int64_t n = (int64_t)e.numel_less_1 + 1, tile = blockIdx.x - first;
    const float* const s32 = static_cast<const float*>(src);
    const uint16_t* const s16 = static_cast<const uint16_t*>(src);
    float* const d32 = static_cast<float*>(dst);
    uint16_t* const d16 = static_cast<uint16_t*>(dst);
    if (bf16 & 1) {
        if (bf16 & 2) clip_tile(s16, d16, n, tile, b.scale, coef);
        else clip_tile(s16, d32, n, tile, b.scale, coef);
    } else {
        if (bf16 & 2) clip_tile(s32, d16, n, tile, b.scale, coef);
        else clip_tile(s32, d32, n, tile, b.scale, coef);
    }
}

}  // namespace

int64_t mixed_tile_elems(int bf16) { return bf16 ? kNormTile<true> : kNormTile<false>; }

hipError_t launch_norms(const NormBatch& b, bool keep, int64_t tiles, float scale, double* partials, hipStream_t stream) {
    const dim3 grid((unsigned)tiles), block(kBlock);
    if (keep) hipLaunchKernelGGL((norms_kernel<true>), grid, block, kNormLds, stream, b, scale, partials);
    else hipLaunchKernelGGL((norms_kernel<false>), grid, block, kNormLds, stream, b, scale, partials);
    return hipGetLastError();
}

hipError_t launch_tensor_sums(const TensorSums& b, hipStream_t stream) {
    hipLaunchKernelGGL(tensor_sums_kernel, dim3(b.count), dim3(kBlock), 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_few_sums(const TensorSums& b, double* out, hipStream_t stream) {
    hipLaunchKernelGGL(few_sums_kernel, dim3(1), dim3(kFewThreads), 0, stream, b, out);
    return hipGetLastError();
}

hipError_t launch_total(const double* norms, int64_t count, double* out, hipStream_t stream) {
    hipLaunchKernelGGL(total_kernel, dim3(1), dim3(kBlock), 0, stream, norms, count, out);
    return hipGetLastError();
}

hipError_t launch_clip(const ClipBatch& b, int64_t tiles, hipStream_t stream) {
    hipLaunchKernelGGL(clip_kernel, dim3((unsigned)tiles), dim3(kBlock), 0, stream, b);
    return hipGetLastError();
}

}  // namespace zs
