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
#include "norm_tile.h"

namespace zs {
namespace {

template <bool BF16, bool KEEP>
__global__ __launch_bounds__(kBlock) void norm_tensors_kernel(const NormBatch b, float scale,
                                                              double* __restrict__ partials) {
    using T = typename GradType<BF16>::T;
    uint32_t first;
    const uint32_t t = find_tensor(b.tab, blockIdx.x, first);
    const NormEntry e = b.e[t];
    const T* const grad = unpack_ptr<const T>(e.lo, e.hi_tail) + (int64_t)(blockIdx.x - first) * kNormTile<BF16>;
    const bool last = blockIdx.x + 1 == b.tab.start[t + 1];
    const int n = last ? (int)(e.hi_tail >> 16) + 1 : (int)kNormTile<BF16>;   // the tile's elements
    const double total = block_sum(norm_tile<BF16, KEEP>(grad, n, last, (e.lo & 2) != 0, scale));
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

int64_t norm_tile_elems(int grad_bf16) { return grad_bf16 ? kNormTile<true> : kNormTile<false>; }

template <bool BF16>
static void launch(const NormBatch& b, bool keep, int64_t tiles, float scale, double* partials, hipStream_t stream) {
    static_assert(kLaunchElems % kNormTile<BF16> == 0, "pieces of a tensor keep its tiles");
    const dim3 grid((unsigned)tiles), block(kBlock);
    if (keep) hipLaunchKernelGGL((norm_tensors_kernel<BF16, true>), grid, block, kNormLds, stream, b, scale, partials);
    else hipLaunchKernelGGL((norm_tensors_kernel<BF16, false>), grid, block, kNormLds, stream, b, scale, partials);
}

hipError_t launch_norm_tensors(const NormBatch& b, int grad_bf16, bool keep, int64_t tiles, float scale,
                               double* partials, hipStream_t stream) {
    if (grad_bf16) launch<true>(b, keep, tiles, scale, partials, stream);
    else launch<false>(b, keep, tiles, scale, partials, stream);
    return hipGetLastError();
}

}  // namespace zs
