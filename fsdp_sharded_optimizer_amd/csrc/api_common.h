// Host-side checks and scalars shared by the C-ABI entry points (internal).
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/zshard.h"
#include "zs_common.h"

namespace zs {

extern thread_local int32_t g_last_hip_error;   // of the last ZS_EHIP on this thread

inline int32_t hip_status(hipError_t e) {
    if (e == hipSuccess) return ZS_OK;
    g_last_hip_error = (int32_t)e;
    return ZS_EHIP;
}

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
inline bool aligned(const void* p, uintptr_t a) { return (addr(p) & (a - 1)) == 0; }

// [p, p+bytes) and [q, q+qbytes) share a byte (empty ranges never overlap)
inline bool overlap(const void* p, int64_t bytes, const void* q, int64_t qbytes) {
    if (bytes <= 0 || qbytes <= 0) return false;
    const uintptr_t a = addr(p), b = addr(q);
    return a < b + (uintptr_t)qbytes && b < a + (uintptr_t)bytes;
}

inline int64_t elem_size(int32_t dtype) { return dtype == ZS_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t d) { return d == ZS_F32 || d == ZS_BF16; }
inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// At most 2^39 elements per call (2 TiB of fp32, beyond any one GPU's
// memory): byte sizes stay far inside int64.  The launchers split a call
// into launches of at most 2^31 elements, so every grid stays below 2^32
// work-items.
constexpr int64_t kMaxElems = int64_t(1) << 39;
inline bool size_ok(int64_t n) { return n >= 0 && n <= kMaxElems; }

inline int32_t adamw_check_hp(const zs_adamw* hp, int64_t n, const double* norm_sq_dev) {
    if (hp == nullptr || !size_ok(n)) return ZS_EINVAL;
    if (hp->step < 1) return ZS_EINVAL;
    if (!(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0))
        return ZS_EINVAL;
    if (!(hp->eps > 0.0) || !std::isfinite(hp->eps)) return ZS_EINVAL;
    if (!(hp->lr >= 0.0) || !std::isfinite(hp->lr)) return ZS_EINVAL;
    if (!(hp->weight_decay >= 0.0) || !std::isfinite(hp->weight_decay)) return ZS_EINVAL;
    if (!(hp->grad_scale > 0.0) || !std::isfinite(hp->grad_scale)) return ZS_EINVAL;
    if (std::isnan(hp->max_norm) || hp->extra_norm_sq < 0.0) return ZS_EINVAL;
    if (norm_sq_dev != nullptr && !aligned(norm_sq_dev, 8)) return ZS_EINVAL;
    return ZS_OK;
}

// host scalars: binary64, each rounded to binary32 once
inline AdamwScalars make_scalars(const zs_adamw* hp) {
    const double t = (double)hp->step;
    const double bias_correction1 = 1.0 - std::pow(hp->beta1, t);
    const double bias_correction2 = 1.0 - std::pow(hp->beta2, t);
    AdamwScalars c;
    std::memset(&c, 0, sizeof(c));
    c.beta1 = (float)hp->beta1;
    c.beta2 = (float)hp->beta2;
    c.one_minus_beta1 = (float)(1.0 - hp->beta1);
    c.one_minus_beta2 = (float)(1.0 - hp->beta2);
    c.step_size = (float)(hp->lr / bias_correction1);
    c.bias_correction2_sqrt = (float)std::sqrt(bias_correction2);
    c.eps = (float)hp->eps;
    c.decay = (float)(1.0 - hp->lr * hp->weight_decay);
    c.grad_scale = (float)hp->grad_scale;
    c.clip = hp->max_norm > 0.0 ? 1 : 0;
    c.max_norm = hp->max_norm;
    c.extra_norm_sq = hp->extra_norm_sq;
    return c;
}

}  // namespace zs
