// C-ABI entry points over lists of tensors (include/zshard_tensors.h):
// validation on the host, then launches of as many tensors as their tables hold.
#include <cstddef>

#include "../../include/zshard_tensors.h"
#include "lists.h"
#include "q8.h"
#include "reduce.h"

using namespace zs;

static_assert(ZS_Q8_BLOCK == kQ8Block, "block length of the header and the kernels");
static_assert(sizeof(zs_adamw_q8_scalars) == sizeof(Q8Scalars) &&
                  offsetof(zs_adamw_q8_scalars, key) == offsetof(Q8Scalars, key), "scalar layout");
static_assert(kLaunchElems % kQ8Pad == 0 && kLaunchElems % kListTile == 0, "pieces start on a tile");

namespace {

// Elements that tile 0 starts before a tensor's first one, so that the moments'
// tiles (most of the bytes) start on whole tiles, 1 KiB, and with them every
// stream at the same offset in elements (views of flat buffers).  405M fp32
// parameters with re-casts, 32 / 33 / 128 elements off: 1687 / 1707 / 1685 us, with
// cache lines alone 1764 / 1843 / 1800 (aligned 1692).  Moments that do not share
// their offset from a cache line: the parameter's.
constexpr int64_t kLine = 128;
int64_t tile_shift(const zs_adamw_tensor& t, int64_t psz) {
    const uintptr_t m = addr(t.exp_avg) / 4, v = addr(t.exp_avg_sq) / 4;
    return (int64_t)(m % 32 == v % 32 ? m : addr(t.param) / (uintptr_t)psz) % kListTile;
}

// Counts the elements whose tiles start off a cache line in some stream: lists
// of which they are the most run differently (tile_in_runs, residency, caching).
struct OffLine {
    int64_t elems = 0;
    // the addresses of the tiles' start, as bits of them all
    void add(int64_t numel, uintptr_t a) {
        if (a % kLine != 0) elems += numel;
    }
    bool most_of(int64_t total) const { return elems > total / 2; }
};

// Whether b's elements come right after a's first n in every stream: the update
// knows no tensors, so the two are one entry then (views of flat buffers: 25M
// bf16 parameters in 290 tensors back to back, one launch instead of three).
bool follows(const zs_adamw_tensor& a, int64_t n, const zs_adamw_tensor& b, int64_t psz, int64_t gsz) {
    return b.param == advance(a.param, n * psz) && b.grad == advance(a.grad, n * gsz) && b.exp_avg == a.exp_avg + n &&
           b.exp_avg_sq == a.exp_avg_sq + n && b.param_bf16 == advance(a.param_bf16, n * 2);
}

int32_t step_tensors(const zs_adamw* hp, const zs_adamw_scalars* sc_dev, const zs_adamw_tensor* list, int32_t count,
                     int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev, void* hip_stream) {
    const int64_t total = list_total(list, count);
    if (total < 0 || !dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return ZS_EINVAL;
    if (sc_dev == nullptr) {
        const int32_t rc = adamw_check_hp(hp, total, norm_sq_dev);
        if (rc != ZS_OK) return rc;
    } else if (!aligned(sc_dev, 8) || (norm_sq_dev != nullptr && !aligned(norm_sq_dev, 8))) {
        return ZS_EINVAL;
    }
    const int64_t psz = elem_size(param_dtype), gsz = elem_size(grad_dtype);
    Ranges ranges;
    OffLine off_line;
    if (!ranges.reserve(count, 5)) return ZS_EINVAL;
    for (int32_t k = 0; k < count; ++k) {
        const zs_adamw_tensor& t = list[k];
        if (t.numel == 0) continue;
        if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr) return ZS_EINVAL;
        if (!aligned(t.param, (uintptr_t)psz) || !aligned(t.grad, (uintptr_t)gsz) || !aligned(t.exp_avg, 4) ||
            !aligned(t.exp_avg_sq, 4))
            return ZS_EINVAL;
        if (t.param_bf16 != nullptr && (param_dtype == ZS_BF16 || !aligned(t.param_bf16, 2))) return ZS_EINVAL;
        if (!packable(t.param) || !packable(t.grad) || !packable(t.exp_avg) || !packable(t.exp_avg_sq) ||
            !packable(t.param_bf16))
            return ZS_EINVAL;
        ranges.add(0, t.param, t.numel * psz, true);
        ranges.add(1, t.grad, t.numel * gsz, false);
        ranges.add(2, t.exp_avg, t.numel * 4, true);
        ranges.add(3, t.exp_avg_sq, t.numel * 4, true);
        ranges.add(4, t.param_bf16, t.numel * 2, true);
        const uintptr_t shift = (uintptr_t)tile_shift(t, psz);
        off_line.add(t.numel, (addr(t.param) - shift * (uintptr_t)psz) | (addr(t.grad) - shift * (uintptr_t)gsz) |
                                  (addr(t.exp_avg) - shift * 4) | (addr(t.exp_avg_sq) - shift * 4) |
                                  (t.param_bf16 == nullptr ? 0 : addr(t.param_bf16) - shift * 2));
    }
    ranges.add_read(norm_sq_dev, 8);
    ranges.add_read(sc_dev, (int64_t)sizeof(zs_adamw_scalars));
    if (ranges.clash()) return ZS_EOVERLAP;

    AdamwBatch b;
    std::memset(&b, 0, sizeof(b));
    if (sc_dev == nullptr) b.sc = make_scalars(hp);
    const bool off = off_line.most_of(total), keep = off || keep_grads(total * gsz);
    b.sc_dev = reinterpret_cast<const AdamwScalars*>(sc_dev);
    b.norm_sq = norm_sq_dev;
    auto launch = [&](const AdamwBatch& x, int64_t tiles) {
        return launch_adamw_tensors(x, param_dtype == ZS_BF16, grad_dtype == ZS_BF16, keep, off, tiles,
                                    as_stream(hip_stream));
    };
    Filler<AdamwBatch, decltype(launch)> fill(b, launch);
    for (int32_t k = 0; k < count; ++k) {
        const zs_adamw_tensor& t = list[k];
        int64_t numel = t.numel;
        if (numel == 0) continue;
        while (k + 1 < count && (list[k + 1].numel == 0 || follows(t, numel, list[k + 1], psz, gsz)))
            numel += list[++k].numel;
        const int64_t shift = tile_shift(t, psz);
        for (int64_t off = 0; off < numel; off += kLaunchElems) {
            const int64_t n = launch_piece(numel, off);
            int at = 0;
            const int32_t rc = fill.add(ceil_div(n + shift, kListTile), at);
            if (rc != ZS_OK) return rc;
            const void* const ptr[5] = {advance(t.param, off * psz), advance(t.grad, off * gsz), t.exp_avg + off,
                                        t.exp_avg_sq + off, advance(t.param_bf16, off * 2)};
            AdamwEntry& e = b.e[at];
            for (int j = 0; j < 5; ++j) e.lo[j] = ptr_lo(ptr[j]);
            e.hi[0] = ptr_hi(ptr[0]) | ptr_hi(ptr[1]) << 16;
            e.hi[1] = ptr_hi(ptr[2]) | ptr_hi(ptr[3]) << 16;
            e.hi[2] = ptr_hi(ptr[4]) | (uint32_t)shift << 16;
            e.numel = (uint32_t)n;
        }
    }
    return fill.flush();
}

uint32_t q8_key(uint32_t seed, int64_t step) { return q8_mix(q8_mix(seed) + (uint32_t)step); }

// The records of the tensors of a call, one after the other: `a` and `b` advance by
// their element sizes, `copy` by 2 bytes.  numel 0: a record without tiles.
template <typename Fill>
class Q8Records {
public:
    Q8Records(Q8Batch& b, Fill& fill) : b_(b), fill_(fill) {}
    int32_t add(int32_t index, void* state, int64_t numel, const void* a, int64_t asz, const void* b, int64_t bsz,
                const void* copy) {
        const bool pieces = numel > kLaunchElems;
        int64_t off = 0;
        do {
            const int64_t n = launch_piece(numel, off);
            const void* const ptr[4] = {advance(a, off * asz), advance(b, off * bsz), state, advance(copy, off * 2)};
            uint32_t top = 0, has = 0;
            for (int j = 0; j < 4 && n > 0; ++j)
                if (ptr[j] != nullptr) top |= (ptr_hi(ptr[j]) >> 8) << (8 * j), has |= 0xFFu << (8 * j);
            // another window of addresses, or a piece before or after
            if (pieces || b_.padded != 0 || ((b_.top ^ top) & has & known_) != 0) {
                const int32_t rc = fill_.flush();
                if (rc != ZS_OK) return rc;
            }
            int at = 0;
            const int32_t rc = fill_.add(ceil_div(n, kQ8Pad), at);
            if (rc != ZS_OK) return rc;
            if (at == 0) {
                known_ = b_.top = 0;
                b_.index = (uint32_t)index;
                b_.off = (uint32_t)(off / kLaunchElems);
                b_.padded = pieces ? (uint32_t)(q8_padded(numel) / kQ8Pad) : 0;
            }
            b_.top |= top;
            known_ |= has;
            Q8Entry& e = b_.e[at];
            e.hi = 0;
            for (int j = 0; j < 4; ++j) {
                e.lo[j] = ptr_lo(ptr[j]);
                e.hi |= (ptr_hi(ptr[j]) & 0xFFu) << (8 * j);
            }
            const uint32_t tail = (uint32_t)(n > 0 ? (n - 1) % kQ8Pad : 0) | (a != nullptr ? kQ8Has0 : 0) |
                                  (b != nullptr ? kQ8Has1 : 0) | (copy != nullptr ? kQ8Has3 : 0);
            uint32_t& word = b_.tail[at / 2];
            word = at % 2 == 0 ? tail : (word & 0xFFFFu) | tail << 16;
            off += kLaunchElems;
        } while (off < numel);
        return ZS_OK;
    }

private:
    Q8Batch& b_;
    Fill& fill_;
    uint32_t known_ = 0;   // the bytes of b_.top that a record of this launch has set
};

int32_t step_tensors_q8(const zs_adamw* hp, uint32_t seed, const zs_adamw_q8_scalars* sc_dev,
                        const zs_adamw_q8_tensor* list, int32_t count, int32_t param_dtype, int32_t grad_dtype,
                        const double* norm_sq_dev, void* hip_stream) {
    const int64_t total = list_total(list, count);
    if (total < 0 || !dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return ZS_EINVAL;
    if (sc_dev == nullptr) {
        const int32_t rc = adamw_check_hp(hp, total, norm_sq_dev);
        if (rc != ZS_OK) return rc;
    } else if (!aligned(sc_dev, 8) || (norm_sq_dev != nullptr && !aligned(norm_sq_dev, 8))) {
        return ZS_EINVAL;
    }
    const int64_t psz = elem_size(param_dtype), gsz = elem_size(grad_dtype);
    Ranges ranges;
    OffLine off_line;
    if (!ranges.reserve(count, 4)) return ZS_EINVAL;
    for (int32_t k = 0; k < count; ++k) {
        const zs_adamw_q8_tensor& t = list[k];
        if (t.numel == 0) continue;
        if (t.param == nullptr || t.grad == nullptr || t.state_q8 == nullptr) return ZS_EINVAL;
        if (!aligned(t.param, (uintptr_t)psz) || !aligned(t.grad, (uintptr_t)gsz) || !aligned(t.state_q8, 16))
            return ZS_EINVAL;
        if (t.param_bf16 != nullptr && (param_dtype == ZS_BF16 || !aligned(t.param_bf16, 2))) return ZS_EINVAL;
        if (!packable(t.param) || !packable(t.grad) || !packable(t.state_q8) || !packable(t.param_bf16)) return ZS_EINVAL;
        ranges.add(0, t.param, t.numel * psz, true);
        ranges.add(1, t.grad, t.numel * gsz, false);
        ranges.add(2, t.state_q8, moments_q8_bytes(t.numel), true);
        ranges.add(3, t.param_bf16, t.numel * 2, true);
        off_line.add(t.numel, addr(t.param) | addr(t.param_bf16));
    }
    ranges.add_read(norm_sq_dev, 8);
    ranges.add_read(sc_dev, (int64_t)sizeof(zs_adamw_q8_scalars));
    if (ranges.clash()) return ZS_EOVERLAP;

    Q8Batch b;
    std::memset(&b, 0, sizeof(b));
    if (sc_dev == nullptr) {
        b.sc.adamw = make_scalars(hp);
        b.sc.key = q8_key(seed, hp->step);
    }
    b.runs = off_line.most_of(total);
    const bool keep = keep_grads(total * gsz);
    b.sc_dev = reinterpret_cast<const Q8Scalars*>(sc_dev);
    b.norm_sq = norm_sq_dev;
    auto launch = [&](const Q8Batch& x, int64_t tiles) {
        return launch_adamw_q8(x, param_dtype == ZS_BF16, grad_dtype == ZS_BF16, keep, tiles, as_stream(hip_stream));
    };
    Filler<Q8Batch, decltype(launch)> fill(b, launch);
    Q8Records<decltype(fill)> records(b, fill);
    for (int32_t k = 0; k < count; ++k) {
        const zs_adamw_q8_tensor& t = list[k];
        const int32_t rc = records.add(k, t.state_q8, t.numel, t.param, psz, t.grad, gsz, t.param_bf16);
        if (rc != ZS_OK) return rc;
    }
    return fill.flush();
}

// both conversions: encode reads the moments and writes the state, decode the reverse
int32_t convert_q8(const zs_moments_q8* list, int32_t count, int32_t dtype, bool encode, uint32_t seed,
                   void* hip_stream) {
    const int64_t total = list_total(list, count);
    if (total < 0 || !dtype_ok(dtype)) return ZS_EINVAL;
    const int64_t sz = elem_size(dtype);
    Ranges ranges;
    OffLine off_line;
    if (!ranges.reserve(count, 3)) return ZS_EINVAL;
    for (int32_t k = 0; k < count; ++k) {
        const zs_moments_q8& t = list[k];
        if (t.numel == 0) continue;
        if (t.state_q8 == nullptr || !aligned(t.state_q8, 16)) return ZS_EINVAL;
        if (!aligned(t.exp_avg, (uintptr_t)sz) || !aligned(t.exp_avg_sq, (uintptr_t)sz)) return ZS_EINVAL;
        if (!packable(t.exp_avg) || !packable(t.exp_avg_sq) || !packable(t.state_q8)) return ZS_EINVAL;
        ranges.add(0, t.exp_avg, t.numel * sz, !encode);
        ranges.add(1, t.exp_avg_sq, t.numel * sz, !encode);
        ranges.add(2, t.state_q8, moments_q8_bytes(t.numel), encode);
        off_line.add(t.numel, addr(t.exp_avg) | addr(t.exp_avg_sq));
    }
    if (ranges.clash()) return ZS_EOVERLAP;
    Q8Batch b;
    std::memset(&b, 0, sizeof(b));
    b.runs = !encode && off_line.most_of(total);
    b.sc.key = q8_key(seed, 0);
    auto launch = [&](const Q8Batch& x, int64_t tiles) {
        return encode ? launch_q8_encode(x, dtype == ZS_BF16, tiles, as_stream(hip_stream))
                      : launch_q8_decode(x, dtype == ZS_BF16, tiles, as_stream(hip_stream));
    };
    Filler<Q8Batch, decltype(launch)> fill(b, launch);
    Q8Records<decltype(fill)> records(b, fill);
    for (int32_t k = 0; k < count; ++k) {
        const zs_moments_q8& t = list[k];
        const bool skip = !encode && t.exp_avg == nullptr && t.exp_avg_sq == nullptr;
        const int32_t rc = records.add(k, t.state_q8, skip ? 0 : t.numel, t.exp_avg, sz, t.exp_avg_sq, sz, nullptr);
        if (rc != ZS_OK) return rc;
    }
    return fill.flush();
}

// partials of the whole list, tensor after tensor; -1 for a bad list
int64_t norm_partials_of(const zs_tensor* grads, int32_t count, int32_t grad_dtype) {
    if (list_total(grads, count) < 0 || !dtype_ok(grad_dtype)) return -1;
    const int64_t tile = norm_tile_elems(grad_dtype == ZS_BF16);
    int64_t parts = 0;
    for (int32_t k = 0; k < count; ++k) parts += ceil_div(grads[k].numel, tile);
    return parts;
}

}  // namespace

extern "C" {

int64_t grad_norm_sq_tensors_workspace_bytes(const zs_tensor* grads, int32_t count, int32_t grad_dtype) {
    const int64_t parts = norm_partials_of(grads, count, grad_dtype);
    if (parts < 0) return -1;
    // only more than kListSumOneGroup partials use the stage; for fewer the size stays the one that programs
    // have asked for so far
    return (parts <= kSumOneGroup ? parts : parts + kReduceChunks) * (int64_t)sizeof(double);
}

int32_t grad_norm_sq_tensors(const zs_tensor* grads, int32_t count, int32_t grad_dtype, double grad_scale,
                             double* out_sq_dev, void* workspace, int64_t workspace_bytes, void* hip_stream) {
    const int64_t parts = norm_partials_of(grads, count, grad_dtype);
    if (parts < 0 || out_sq_dev == nullptr || !aligned(out_sq_dev, 8)) return ZS_EINVAL;
    if (!(grad_scale > 0.0) || !std::isfinite(grad_scale)) return ZS_EINVAL;
    const int64_t gsz = elem_size(grad_dtype);
    const int64_t need = grad_norm_sq_tensors_workspace_bytes(grads, count, grad_dtype);
    if (need > 0 && (workspace == nullptr || !aligned(workspace, 8))) return ZS_EINVAL;
    if (workspace_bytes < need) return ZS_EWORKSPACE;
    // only the workspace and *out_sq_dev are written
    if (overlap(out_sq_dev, 8, workspace, need)) return ZS_EOVERLAP;
    bool clash = false;
    for (int32_t k = 0; k < count; ++k) {
        const zs_tensor& t = grads[k];
        if (t.numel == 0) continue;
        if (t.ptr == nullptr || !aligned(t.ptr, (uintptr_t)gsz) || !packable(t.ptr)) return ZS_EINVAL;
        clash = clash || overlap(t.ptr, t.numel * gsz, out_sq_dev, 8) || overlap(t.ptr, t.numel * gsz, workspace, need);
    }
    if (clash) return ZS_EOVERLAP;

    double* const partials = static_cast<double*>(workspace);
    int64_t done = 0;   // partials of the launches before
    NormBatch b;
    std::memset(&b, 0, sizeof(b));
    const bool keep = keep_grads(list_total(grads, count) * gsz);
    auto launch = [&](const NormBatch& x, int64_t tiles) {
        // a list of one tile: its partial is the result
        const hipError_t e = launch_norm_tensors(x, grad_dtype == ZS_BF16, keep, tiles, (float)grad_scale,
                                                 parts == 1 ? out_sq_dev : partials + done, as_stream(hip_stream));
        done += tiles;
        return e;
    };
    Filler<NormBatch, decltype(launch)> fill(b, launch);
    const int64_t tile = norm_tile_elems(grad_dtype == ZS_BF16);
    for (int32_t k = 0; k < count; ++k)
        for (int64_t off = 0; off < grads[k].numel; off += kLaunchElems) {
            const int64_t n = launch_piece(grads[k].numel, off);
            int at = 0;
            const int32_t rc = fill.add(ceil_div(n, tile), at);
            if (rc != ZS_OK) return rc;
            const void* const p = advance(grads[k].ptr, off * gsz);
            b.e[at] = NormEntry{ptr_lo(p), ptr_hi(p) | (uint32_t)((n - 1) % tile) << 16};
        }
    const int32_t rc = fill.flush();
    if (rc != ZS_OK || parts == 1) return rc;
    return hip_status(launch_list_sum(partials, parts, partials + parts, out_sq_dev, as_stream(hip_stream)));
}

int32_t adamw_step_tensors(const zs_adamw* hp, const zs_adamw_tensor* tensors, int32_t count, int32_t param_dtype,
                           int32_t grad_dtype, const double* norm_sq_dev, void* hip_stream) {
    if (hp == nullptr) return ZS_EINVAL;
    return step_tensors(hp, nullptr, tensors, count, param_dtype, grad_dtype, norm_sq_dev, hip_stream);
}

int32_t adamw_step_tensors_dev(const zs_adamw_scalars* scalars_dev, const zs_adamw_tensor* tensors, int32_t count,
                               int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev, void* hip_stream) {
    if (scalars_dev == nullptr) return ZS_EINVAL;
    return step_tensors(nullptr, scalars_dev, tensors, count, param_dtype, grad_dtype, norm_sq_dev, hip_stream);
}

int64_t moments_q8_bytes(int64_t n) {
    if (!size_ok(n)) return -1;
    const int64_t p = q8_padded(n);
    return ceil_div(2 * p + p / (kQ8Block / 2), kLine) * kLine;
}

int32_t moments_q8_encode(const zs_moments_q8* moments, int32_t count, int32_t dtype, uint32_t seed,
                          void* hip_stream) {
    return convert_q8(moments, count, dtype, true, seed, hip_stream);
}

int32_t moments_q8_decode(const zs_moments_q8* moments, int32_t count, int32_t dtype, void* hip_stream) {
    return convert_q8(moments, count, dtype, false, 0, hip_stream);
}

int32_t adamw_step_tensors_q8(const zs_adamw* hp, uint32_t seed, const zs_adamw_q8_tensor* tensors, int32_t count,
                              int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev, void* hip_stream) {
    if (hp == nullptr) return ZS_EINVAL;
    return step_tensors_q8(hp, seed, nullptr, tensors, count, param_dtype, grad_dtype, norm_sq_dev, hip_stream);
}

int32_t adamw_q8_scalars(const zs_adamw* hp, uint32_t seed, zs_adamw_q8_scalars* out) {
    if (out == nullptr) return ZS_EINVAL;
    const int32_t rc = adamw_scalars(hp, &out->adamw);
    if (rc != ZS_OK) return rc;
    out->key = q8_key(seed, hp->step);
    out->reserved = 0;
    return ZS_OK;
}

int32_t adamw_step_tensors_q8_dev(const zs_adamw_q8_scalars* scalars_dev, const zs_adamw_q8_tensor* tensors,
                                  int32_t count, int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev,
                                  void* hip_stream) {
    if (scalars_dev == nullptr) return ZS_EINVAL;
    return step_tensors_q8(nullptr, 0, scalars_dev, tensors, count, param_dtype, grad_dtype, norm_sq_dev, hip_stream);
}

}  // extern "C"
