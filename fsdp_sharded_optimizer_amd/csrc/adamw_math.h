// The AdamW arithmetic of one element and the clip coefficient (device),
// shared by the steps over a flat shard and over lists of tensors (internal).
#pragma once

#include "zs_common.h"

namespace zs {

// One element: the moments in place and the returned step u, in the order
// and with the roundings the header documents.  Built with
// -ffp-contract=off: no multiply-add fusion; the quotient and square root
// are IEEE round-to-nearest (correctly rounded fp32 division and sqrt are
// requested at compile time).
__device__ __forceinline__ float adam_elem(const AdamwScalars& a, float coef, float gr, float& m, float& v) {
    float g = gr * a.grad_scale;
    g = g * coef;
    const float m_keep = a.beta1 * m;
    const float m_new = a.one_minus_beta1 * g;
    m = m_keep + m_new;
    const float g2 = g * g;
    const float v_keep = a.beta2 * v;
    const float v_new = a.one_minus_beta2 * g2;
    v = v_keep + v_new;
    const float root = sqrtf(v);
    float den = root / a.bias_correction2_sqrt;
    den = den + a.eps;
    const float ratio = m / den;
    return ratio * a.step_size;
}

// the parameter after the step: decoupled decay, then the step
__device__ __forceinline__ float apply_step(const AdamwScalars& a, float p, float u) {
    const float pd = p * a.decay;
    return pd - u;
}

// Clip coefficient from the squared norm, in binary64 (uniform per wave).
// Returns false when the global squared norm is not finite: the step is
// skipped, no state is written (the update form writes -0.0, see below).
__device__ __forceinline__ bool clip_coef(const AdamwScalars& a, const double* norm_sq, float& coef) {
    coef = 1.0f;
    if (norm_sq == nullptr) return true;
    const double s = *norm_sq + a.extra_norm_sq;
    if (!__builtin_isfinite(s)) return false;
    if (a.clip) {
        const double total = sqrt(s);
        double c = a.max_norm / (total + 1e-6);
        if (c > 1.0) c = 1.0;
        coef = (float)c;
    }
    return true;
}

}  // namespace zs
