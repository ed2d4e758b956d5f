// C-ABI entry points over lists of mixed precision (include/zshard_tensors.h):
// validation on the host, then launches of as many tensors as their tables hold.
#include "../../include/zshard_tensors.h"
#include "clip.h"
#include "lists.h"

using namespace zs;

namespace {

// one tensor's tiles are workgroups of one launch
constexpr int64_t kMaxTensorElems = int64_t(1) << 35;

int64_t mixed_tiles(const zs_mixed_tensor& t) { return ceil_div(t.numel, mixed_tile_elems(t.dtype == ZS_BF16)); }

// partials of the whole list; -1 for a bad one
int64_t mixed_partials(const zs_mixed_tensor* list, int32_t count) {
    if (list_total(list, count) < 0) return -1;
    int64_t parts = 0;
    for (int32_t k = 0; k < count; ++k) {
        if (!dtype_ok(list[k].dtype) || list[k].reserved != 0 || list[k].numel > kMaxTensorElems) return -1;
        parts += mixed_tiles(list[k]);
    }
    return parts;
}

bool pointer_ok(const zs_mixed_tensor& t) {
    return t.ptr != nullptr && aligned(t.ptr, (uintptr_t)elem_size(t.dtype)) && packable(t.ptr);
}

}  // namespace

extern "C" {

int64_t grad_norms_sq_tensors_workspace_bytes(const zs_mixed_tensor* grads, int32_t count) {
    const int64_t parts = mixed_partials(grads, count);
    return parts < 0 ? -1 : (parts + count) * (int64_t)sizeof(double);
}

int32_t grad_norms_sq_tensors(const zs_mixed_tensor* grads, int32_t count, double grad_scale, double* norms_sq_dev,
                              double* out_sq_dev, void* workspace, int64_t workspace_bytes, void* hip_stream) {
    const int64_t parts = mixed_partials(grads, count);
    if (parts < 0 || out_sq_dev == nullptr || !aligned(out_sq_dev, 8) || !aligned(norms_sq_dev, 8)) return ZS_EINVAL;
    if (!positive_float(grad_scale)) return ZS_EINVAL;
    const int64_t need = grad_norms_sq_tensors_workspace_bytes(grads, count);
    if (need > 0 && (workspace == nullptr || !aligned(workspace, 8))) return ZS_EINVAL;
    if (workspace_bytes < need) return ZS_EWORKSPACE;
    Ranges ranges;   // gradients may overlap one another
    if (!ranges.reserve(std::max(count, 3), 2)) return ZS_EINVAL;
    int64_t bytes = 0;
    for (int32_t k = 0; k < count; ++k) {
        if (grads[k].numel == 0) continue;
        if (!pointer_ok(grads[k])) return ZS_EINVAL;
        ranges.add(0, grads[k].ptr, grads[k].numel * elem_size(grads[k].dtype), false);
        bytes += grads[k].numel * elem_size(grads[k].dtype);
    }
    ranges.add(1, workspace, need, true);
    ranges.add(1, out_sq_dev, 8, true);
    ranges.add(1, norms_sq_dev, (int64_t)count * 8, true);
    if (ranges.clash()) return ZS_EOVERLAP;

    double* partials = static_cast<double*>(workspace);
    double* const norms = norms_sq_dev != nullptr ? norms_sq_dev : partials + parts;
    const hipStream_t stream = as_stream(hip_stream);
    NormBatch b;
    std::memset(&b, 0, sizeof(b));
    const bool keep = keep_grads(bytes);
    auto launch = [&](const NormBatch& x, int64_t tiles) {
        return launch_norms(x, keep, tiles, (float)grad_scale, partials, stream);
    };
    Filler<NormBatch, decltype(launch)> fill(b, launch);
    constexpr int64_t kMost = sizeof(b.e) / sizeof(b.e[0]);
    TensorSums sums;
    std::memset(&sums, 0, sizeof(sums));
    int64_t entries = 0, tiles = 0, done = 0;   // of this launch; tensors of the launches before
    const bool few = count > 0 && count <= kFewTensors && parts <= kFewPartials;   // (one launch)
    auto emit = [&]() -> int32_t {
        int32_t rc = fill.flush();
        if (rc != ZS_OK || sums.count == 0) return rc;
        sums.grid = (uint32_t)tiles;
        sums.partials = partials;
        sums.norms = norms + done;
        if (few) return hip_status(launch_few_sums(sums, out_sq_dev, stream));
        rc = hip_status(launch_tensor_sums(sums, stream));
        partials += tiles;
        done += sums.count;
        sums.count = 0;
        entries = tiles = 0;
        return rc;
    };
    for (int32_t k = 0; k < count; ++k) {
        const zs_mixed_tensor& t = grads[k];
        const int64_t pieces = ceil_div(t.numel, kLaunchElems), more = mixed_tiles(t);
        if (entries + pieces > kMost || tiles + more > kListMaxTiles || sums.count == (uint32_t)kSumsMax) {
            const int32_t rc = emit();
            if (rc != ZS_OK) return rc;
        }
        const int64_t gsz = elem_size(t.dtype), tile = mixed_tile_elems(t.dtype == ZS_BF16);
        for (int64_t off = 0; off < t.numel; off += kLaunchElems) {
            const int64_t n = launch_piece(t.numel, off);
            int at = 0;
            const int32_t rc = fill.add(ceil_div(n, tile), at);
            if (rc != ZS_OK) return rc;
            const void* const p = advance(t.ptr, off * gsz);
            b.e[at] = NormEntry{ptr_lo(p), ptr_hi(p) | (uint32_t)((n - 1) % tile) << 16 | (t.dtype == ZS_BF16 ? kNormBf16 : 0)};
        }
        sums.start[sums.count++] = (uint32_t)tiles;
        tiles += more;
        entries += pieces;
        sums.start[sums.count] = (uint32_t)tiles;
    }
    const int32_t rc = emit();
    if (rc != ZS_OK || few) return rc;
    return hip_status(launch_total(norms, count, out_sq_dev, stream));
}

int32_t grad_clip_tensors(const zs_mixed_tensor* grads, const zs_mixed_tensor* out, int32_t count, double grad_scale,
                          double max_norm, double extra_norm_sq, const double* norm_sq_dev, void* hip_stream) {
    if (mixed_partials(grads, count) < 0 || mixed_partials(out, count) < 0) return ZS_EINVAL;
    if (!positive_float(grad_scale)) return ZS_EINVAL;
    if (std::isnan(max_norm) || !(extra_norm_sq >= 0.0) || !aligned(norm_sq_dev, 8)) return ZS_EINVAL;
    Ranges ranges;
    if (!ranges.reserve(count, 2)) return ZS_EINVAL;
    for (int32_t k = 0; k < count; ++k) {
        const zs_mixed_tensor &g = grads[k], &y = out[k];
        if (g.numel != y.numel) return ZS_EINVAL;
        if (g.numel == 0) continue;
        if (!pointer_ok(g) || !pointer_ok(y)) return ZS_EINVAL;
        // a tensor clipped in place is one that is written
        if (!(g.ptr == y.ptr && g.dtype == y.dtype)) ranges.add(0, g.ptr, g.numel * elem_size(g.dtype), false);
        ranges.add(1, y.ptr, y.numel * elem_size(y.dtype), true);
    }
    ranges.add_read(norm_sq_dev, 8);
    if (ranges.clash()) return ZS_EOVERLAP;

    ClipBatch b;
    std::memset(&b, 0, sizeof(b));
    b.norm_sq = norm_sq_dev;
    b.max_norm = max_norm;
    b.extra_norm_sq = extra_norm_sq;
    b.scale = (float)grad_scale;
    b.clip = max_norm > 0.0;
    auto launch = [&](ClipBatch& x, int64_t tiles) {
        const hipError_t e = launch_clip(x, tiles, as_stream(hip_stream));
        std::memset(x.bf16, 0, sizeof(x.bf16));
        return e;
    };
    Filler<ClipBatch, decltype(launch)> fill(b, launch);
    for (int32_t k = 0; k < count; ++k)
        for (int64_t off = 0; off < grads[k].numel; off += kLaunchElems) {
            const int64_t n = launch_piece(grads[k].numel, off);
            int at = 0;
            const int32_t rc = fill.add(ceil_div(n, kClipTile), at);
            if (rc != ZS_OK) return rc;
            const void* const p = advance(grads[k].ptr, off * elem_size(grads[k].dtype));
            const void* const q = advance(out[k].ptr, off * elem_size(out[k].dtype));
            b.e[at] = ClipEntry{{ptr_lo(p), ptr_lo(q)}, ptr_hi(p) | ptr_hi(q) << 16, (uint32_t)(n - 1)};
            const uint32_t bits = (grads[k].dtype == ZS_BF16 ? 1u : 0u) | (out[k].dtype == ZS_BF16 ? 2u : 0u);
            b.bf16[at / 16] |= bits << (2 * (at % 16));
        }
    return fill.flush();
}

}  // extern "C"
