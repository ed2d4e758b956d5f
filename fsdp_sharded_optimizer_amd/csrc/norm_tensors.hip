// The squared global norm of a list of gradients.
//
// sum (double)fl32(widen(g) * scale)^2 over every tensor, in binary64: each
// workgroup adds the squares of one tile of one tensor (zs::add_squares4, the
// butterfly and LDS order of reduce.h) and writes one partial.  A list of one
// tile has its result then; up to kSumOneGroup = 2048 partials are added by one
// 256-thread workgroup, more than kListSumOneGroup = 16384 by two launches with
// a stage between them (both launch_sum_partials), those between by one
// 1024-thread workgroup (list_sum_kernel).  The association depends only on the
// numels, the dtype and their order.  HBM-bound: 4 (2) bytes per element, read
// once.
//
// Layout: the standalone norm's (norm.hip): 256-thread workgroups, four
// lane-contiguous 128-bit loads per lane (4096 fp32 or 8192 bf16 elements),
// all issued before the first square, 24 KiB of LDS reserved (6 workgroups
// per CU).  The gradients are only read, so they are loaded 128 bits wide at
// any element alignment.
#include "reduce.h"
#include "tensors.h"

namespace zs {
namespace {

constexpr int kQ = 4;
constexpr unsigned kLds = 24576;
template <bool BF16> constexpr int kVec = BF16 ? 8 : 4;   // elements of a 128-bit load
template <bool BF16> constexpr int64_t kTile = (int64_t)kBlock * kVec<BF16> * kQ;

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

template <bool BF16, bool KEEP>
__global__ __launch_bounds__(kBlock) void norm_tensors_kernel(const NormBatch b, float scale,
                                                              double* __restrict__ partials) {
    constexpr int VE = kVec<BF16>;
    using T = typename GradType<BF16>::T;
    uint32_t first;
    const uint32_t t = find_tensor(b.tab, blockIdx.x, first);
    const NormEntry e = b.e[t];
    const T* const grad = unpack_ptr<const T>(e.lo, e.hi_tail) + (int64_t)(blockIdx.x - first) * kTile<BF16>;
    const bool last = blockIdx.x + 1 == b.tab.start[t + 1];
    const int n = last ? (int)(e.hi_tail >> 16) + 1 : (int)kTile<BF16>;   // the tile's elements
    const int lane0 = threadIdx.x * VE;
    u32x4 v[kQ];
    if (BF16 && (e.lo & 2) && !last) {
        // bf16 at an odd offset: a lane's 16 bytes would span 5 words.  The words
        // from its second element on instead; its first element is in the last
        // word of the lane before (of a wave's first lane: loaded by itself).
        uint32_t head[kQ] = {};
#pragma unroll
        for (int q = 0; q < kQ; ++q) v[q] = ld_u32x4_any<KEEP>(grad + lane0 + q * kBlock * VE + 1);
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) head[q] = (uint32_t)grad[lane0 + q * kBlock * VE] << 16;
        }
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            const u32x4 w = v[q];
            const uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp((int)head[q], (int)w.w, 0x138, 0xF, 0xF, false);   // wave_shr:1
            v[q] = u32x4{__builtin_amdgcn_alignbit(w.x, before, 16), __builtin_amdgcn_alignbit(w.y, w.x, 16),
                         __builtin_amdgcn_alignbit(w.z, w.y, 16), __builtin_amdgcn_alignbit(w.w, w.z, 16)};
        }
    } else if (n == (int)kTile<BF16>) {
#pragma unroll
        for (int q = 0; q < kQ; ++q) v[q] = ld_u32x4_any<KEEP>(grad + lane0 + q * kBlock * VE);
    } else {   // a tensor's ragged last tile: elements past the end add +0
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            const int at = lane0 + q * kBlock * VE;
            if (at + VE <= n) v[q] = ld_u32x4_any<KEEP>(grad + at);
            else v[q] = last_words<BF16>(grad, at, n);
        }
    }
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
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
    const double total = block_sum(s0 + s1);
    if (threadIdx.x == 0) partials[xcd_slot(blockIdx.x, gridDim.x)] = total;
}

// Up to kListSumOneGroup partials in one workgroup, in a fixed order: thread i adds
// the partials i, i + 1024, ..., then the butterfly of its wave, then the waves.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void list_sum_kernel(const double* __restrict__ partials, int count,
                                                               double* __restrict__ out) {
    __shared__ double part[kSumThreads / 64];
    constexpr int kMost = (int)(kListSumOneGroup / kSumThreads);
    double x[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int i = threadIdx.x + k * kSumThreads;
        x[k] = i < count ? partials[i] : 0.0;
    }
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < kMost; ++k) s += x[k];
    s = wave_sum(s);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
#pragma unroll
        for (int w = 0; w < kSumThreads / 64; ++w) s += part[w];
        *out = s;
    }
}

}  // namespace

hipError_t launch_list_sum(const double* partials, int64_t count, double* stage, double* out, hipStream_t stream) {
    if (count <= kSumOneGroup || count > kListSumOneGroup) return launch_sum_partials(partials, count, stage, out, stream);
    hipLaunchKernelGGL(list_sum_kernel, dim3(1), dim3(kSumThreads), 0, stream, partials, (int)count, out);
    return hipGetLastError();
}

int64_t norm_tile_elems(int grad_bf16) { return grad_bf16 ? kTile<true> : kTile<false>; }

template <bool BF16>
static void launch(const NormBatch& b, bool keep, int64_t tiles, float scale, double* partials, hipStream_t stream) {
    static_assert(kLaunchElems % kTile<BF16> == 0, "pieces of a tensor keep its tiles");
    const dim3 grid((unsigned)tiles), block(kBlock);
    if (keep) hipLaunchKernelGGL((norm_tensors_kernel<BF16, true>), grid, block, kLds, stream, b, scale, partials);
    else hipLaunchKernelGGL((norm_tensors_kernel<BF16, false>), grid, block, kLds, stream, b, scale, partials);
}

hipError_t launch_norm_tensors(const NormBatch& b, int grad_bf16, bool keep, int64_t tiles, float scale,
                               double* partials, hipStream_t stream) {
    if (grad_bf16) launch<true>(b, keep, tiles, scale, partials, stream);
    else launch<false>(b, keep, tiles, scale, partials, stream);
    return hipGetLastError();
}

}  // namespace zs
