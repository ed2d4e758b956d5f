// Norms and clipping over lists of mixed precision: the tables that travel in the
// kernel arguments (internal).
#pragma once

#include "tensors.h"

namespace zs {

// A tensor's dtype is the top bit of its NormEntry's tail.
constexpr uint32_t kNormBf16 = 0x80000000u;
int64_t mixed_tile_elems(int bf16);   // elements per workgroup (one binary64 partial each)
hipError_t launch_norms(const NormBatch& b, bool keep, int64_t tiles, float scale, double* partials, hipStream_t stream);

// Where the tensors of one launch of `grid` workgroups have their partials:
// tensor k the workgroups [start[k], start[k + 1]), none where it has no elements.
constexpr int kSumsMax = 960;
struct TensorSums {
    uint32_t start[kSumsMax + 1];
    uint32_t count, grid;
    const double* partials;    // of the launch
    double* norms;             // of the first tensor
};
static_assert(sizeof(TensorSums) <= 4096, "kernel arguments");
hipError_t launch_tensor_sums(const TensorSums& b, hipStream_t stream);
// A list of at most this many tensors and partials in one launch has its sums in one
// more (1M gradients in 12 tensors: 21.0 -> 19.7 us with their clipping).
constexpr int kFewTensors = 64;
constexpr int64_t kFewPartials = 2048;
hipError_t launch_few_sums(const TensorSums& b, double* out, hipStream_t stream);
hipError_t launch_total(const double* norms, int64_t count, double* out, hipStream_t stream);

constexpr int64_t kClipTile = 4096;
struct ClipEntry {
    uint32_t lo[2];            // source, destination
    uint32_t hi;               // source | destination << 16
    uint32_t numel_less_1;
};
struct ClipBatch {
    ListTable<190> tab;
    ClipEntry e[190];
    const double* norm_sq;     // nullable
    double max_norm, extra_norm_sq;
    float scale;
    int32_t clip;
    uint32_t bf16[12];         // two bits an entry: the source's and the destination's dtype
};
static_assert(sizeof(ClipBatch) <= 4096, "kernel arguments");
hipError_t launch_clip(const ClipBatch& b, int64_t tiles, hipStream_t stream);

}  // namespace zs
