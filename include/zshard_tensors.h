/*
 * zshard_tensors.h — the optimizer step over many tensors at once (part of
 * libzshard.so; the conventions, types and error codes are zshard.h's).
 *
 * zshard.h steps one flat shard.  The calls here take a host list of device
 * tensors, as a model that is not flattened has them: the squared gradient
 * norm over the list, the AdamW update of every tensor with its moments in
 * fp32 or in 8 bits, and the conversions of 8-bit moments.  The list is read
 * during the call only: tables of it travel in the kernel arguments (98
 * tensors to a launch, 150 with 8-bit moments, 328 for the norm), so nothing is
 * allocated on the device, copied to it or kept, and a call can be captured into
 * a HIP graph as is.
 *
 * For every call: count >= 0 and the list not NULL with count > 0; a tensor's
 * numel >= 0, the sum at most 2^39; a tensor with numel 0 is skipped (its
 * pointers are not looked at).  Every tensor is contiguous, fp32 pointers are
 * 4-byte and bf16 pointers 2-byte aligned; views at any element offset are
 * fine (full speed: every stream at one common offset, in elements, from a
 * boundary of 256).  A buffer that is written must
 * not overlap any other buffer of the list (ZS_EOVERLAP); buffers that are
 * only read may overlap one another (two tensors may share one gradient).
 */
#ifndef ZSHARD_TENSORS_H
#define ZSHARD_TENSORS_H

#include "zshard.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * grad_norm_sq_tensors_workspace_bytes — bytes of device workspace
 * grad_norm_sq_tensors needs for this list (only the numels are read; 0 for
 * an empty list, -1 for an invalid one).  Host only.
 */
ZS_API int64_t grad_norm_sq_tensors_workspace_bytes(const zs_tensor* grads, int32_t count, int32_t grad_dtype);

/*
 * grad_norm_sq_tensors — the squared global norm of a list of gradients, the
 * norm_sq_dev of the steps below (zshard.h's grad_norm_sq over one buffer).
 * *out_sq_dev = sum over every tensor's elements of (double)g1^2 with g1 =
 * fl32(widen(g) * (float)grad_scale); squares exact in binary64, summed in
 * binary64 in a fixed order that depends only on the numels and grad_dtype:
 * bit-reproducible run to run.  An empty list writes 0.
 * grads: host array of `count` device tensors of grad_dtype (ZS_F32 or
 * ZS_BF16), read; out_sq_dev: device double, written; workspace: device,
 * 8-byte aligned, at least grad_norm_sq_tensors_workspace_bytes bytes, scratch
 * owned by the caller until the stream has passed the call.
 * Errors: ZS_EINVAL, ZS_EWORKSPACE, ZS_EOVERLAP (the workspace or *out_sq_dev
 * with a gradient or one another), ZS_EHIP.
 */
ZS_API int32_t grad_norm_sq_tensors(const zs_tensor* grads, int32_t count, int32_t grad_dtype, double grad_scale,
                                    double* out_sq_dev, void* workspace, int64_t workspace_bytes, void* hip_stream);

/* One tensor of adamw_step_tensors. */
typedef struct {
    void* param;           /* fp32 or bf16 (param_dtype), read-write */
    const void* grad;      /* fp32 or bf16 (grad_dtype), read */
    float* exp_avg;        /* fp32, read-write */
    float* exp_avg_sq;     /* fp32, read-write */
    uint16_t* param_bf16;  /* bf16 re-cast of an fp32 param, written; or NULL */
    int64_t numel;
} zs_adamw_tensor;

/*
 * adamw_step_tensors — the AdamW update of every tensor of a list.
 * Element for element the update of adamw_step (param_dtype ZS_F32: the fp32
 * parameter, with its bf16 re-cast where param_bf16 is not NULL) or of
 * adamw_step_no_master (param_dtype ZS_BF16: the bf16 parameter in place;
 * param_bf16 must be NULL), with the gradient widen(grad): results are bit
 * for bit those of that call on each tensor (its gradient widened to fp32).
 * hp and norm_sq_dev as there: one clip coefficient for the whole list, and a
 * non-finite norm leaves every tensor unchanged.
 * Errors: ZS_EINVAL, ZS_EOVERLAP, ZS_EHIP (lists of more than 98 tensors are
 * several launches: a failed one leaves the earlier ones enqueued).
 */
ZS_API int32_t adamw_step_tensors(const zs_adamw* hp, const zs_adamw_tensor* tensors, int32_t count,
                                  int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev,
                                  void* hip_stream);

/* adamw_step_tensors with its scalars read from device memory when the
 * kernels run (as adamw_step_dev); scalars_dev must not overlap a written
 * buffer. */
ZS_API int32_t adamw_step_tensors_dev(const zs_adamw_scalars* scalars_dev, const zs_adamw_tensor* tensors,
                                      int32_t count, int32_t param_dtype, int32_t grad_dtype,
                                      const double* norm_sq_dev, void* hip_stream);

/*
 * 8-bit moments — both moments of one tensor in one buffer, about 2 bytes per
 * element instead of 8.  The elements are grouped in blocks of
 * ZS_Q8_BLOCK = 256 consecutive ones (a tensor's last block may be shorter),
 * and each block has a power-of-two scale per moment, so scaling is exact.
 * A code is a small binary floating-point number with 3 fraction bits:
 * exp_avg a sign and 4 exponent bits, exp_avg_sq 5 exponent bits.  With M the
 * block's largest magnitude as a binary32 bit pattern,
 *   e = min(255, (M + 0x0FFFFF) >> 23)   (one byte per block and moment)
 *   s = |x| * 2^(T - e), T = 15 (exp_avg) or 31 (exp_avg_sq), in binary32
 *   code = (pattern(s) + r) >> 20   (exp_avg: the sign of x above it;
 *                                    exp_avg_sq: at least 1 for x > 0)
 *   value = +-float(code << 20 as a pattern) * 2^(e - T)
 * so exp_avg spans 5.3 decades below the block's largest value and exp_avg_sq
 * 10.2 (the subnormal codes included), in steps of 6.25-12.5 %.  Rounding is
 * stochastic and unbiased: r is a 20-bit dither.  (To nearest, a second
 * moment at beta2 = 0.999 would hardly ever change: one step moves it by
 * 0.1 %, half a code step is 3-6 %.)  A positive second moment never becomes
 * 0, so no update is divided by eps alone.  A block that holds a non-finite
 * value, or one above 1.875 * 2^127, has e = 255 and reads as NaN.
 * Dither, in 32-bit arithmetic: mix(x): x ^= x >> 16; x *= 0x6A09E667;
 * x ^= x >> 15; x *= 0xBB67AE85; x ^= x >> 16.  A call has a key (below);
 * tensor k of the list key_k = mix(key + k * 0x9E3779B9); element i of it,
 * with G = i / 4,  h = mix(low(G) + high(G) * 0x9E3779B9 + key_k) +
 * (i % 4) * 0x9E3779B9;  r = h >> 12 for exp_avg, h & 0xFFFFF for exp_avg_sq.
 * The order of codes and scales in the buffer is the library's own.  A buffer
 * of zero bytes holds zero moments.  Buffers are 16-byte aligned (full speed:
 * 1 KiB) and hold moments_q8_bytes(numel) bytes.
 */
#define ZS_Q8_BLOCK 256

/* Bytes of the 8-bit moments of n elements (-1 for n < 0 or n > 2^39).  Host only. */
ZS_API int64_t moments_q8_bytes(int64_t n);

/* One tensor of the conversions. */
typedef struct {
    void* exp_avg;         /* fp32 or bf16 (dtype), or NULL */
    void* exp_avg_sq;      /* fp32 or bf16 (dtype), or NULL */
    void* state_q8;        /* 8-bit moments */
    int64_t numel;
} zs_moments_q8;

/*
 * moments_q8_encode — moments into 8 bits, for every tensor of a list.
 * exp_avg, exp_avg_sq: read, of dtype ZS_F32 or ZS_BF16 (NULL: zeros); a
 * negative exp_avg_sq is stored as its magnitude.  state_q8: written, every
 * byte that moments_q8_decode or a step reads.  The key is mix(mix(seed)).
 * Values that came out of moments_q8_decode are kept exactly, whatever the
 * seed: a state saved and loaded goes on bit for bit.
 */
ZS_API int32_t moments_q8_encode(const zs_moments_q8* moments, int32_t count, int32_t dtype, uint32_t seed,
                                 void* hip_stream);

/*
 * moments_q8_decode — the values of 8-bit moments, for every tensor of a
 * list.  state_q8: read; exp_avg, exp_avg_sq: written, of dtype ZS_F32 or
 * ZS_BF16 (NULL: skipped).  A value has 4 significant bits, so fp32 holds it
 * exactly, and bf16 from 2^-130 up (below, its subnormals round to nearest).
 */
ZS_API int32_t moments_q8_decode(const zs_moments_q8* moments, int32_t count, int32_t dtype, void* hip_stream);

/* One tensor of adamw_step_tensors_q8. */
typedef struct {
    void* param;           /* fp32 or bf16 (param_dtype), read-write */
    const void* grad;      /* fp32 or bf16 (grad_dtype), read */
    void* state_q8;        /* 8-bit moments, read-write */
    uint16_t* param_bf16;  /* bf16 re-cast of an fp32 param, written; or NULL */
    int64_t numel;
} zs_adamw_q8_tensor;

/*
 * adamw_step_tensors_q8 — adamw_step_tensors on 8-bit moments: each tensor's
 * moments are decoded, the new ones formed in fp32 as adamw_step forms them
 * (the same operations and roundings), the parameter updated with these, and
 * they are stored in 8 bits.  The parameter's step is within 8 * 2^-24 of the
 * quotient of those moments (formed with the hardware's root and reciprocal
 * where eps times bias correction 2's root is at least 2^-38 and eps below 2^100,
 * elsewhere and in a tensor's last, incomplete 512 elements with IEEE ones).  The key is mix(mix(seed) + step), step the low
 * 32 bits of hp->step: the same call on the same data gives the same bits.
 * A non-finite norm leaves every tensor and its moments unchanged; without a
 * norm a gradient that is not finite makes its whole block's moments NaN.
 * Full speed: param, grad and param_bf16 on boundaries of 256 elements.
 */
ZS_API int32_t adamw_step_tensors_q8(const zs_adamw* hp, uint32_t seed, const zs_adamw_q8_tensor* tensors,
                                     int32_t count, int32_t param_dtype, int32_t grad_dtype,
                                     const double* norm_sq_dev, void* hip_stream);

/* The scalars of one adamw_step_tensors_q8: adamw_scalars' and the key. */
typedef struct {
    zs_adamw_scalars adamw;
    uint32_t key;
    uint32_t reserved;     /* 0 */
} zs_adamw_q8_scalars;

/* The scalars adamw_step_tensors_q8 forms from hp and seed, on the host.
 * Errors as adamw_scalars. */
ZS_API int32_t adamw_q8_scalars(const zs_adamw* hp, uint32_t seed, zs_adamw_q8_scalars* out);

/* adamw_step_tensors_q8 with its scalars read from device memory when the
 * kernels run; scalars_dev (8-byte aligned) must not overlap a written
 * buffer. */
ZS_API int32_t adamw_step_tensors_q8_dev(const zs_adamw_q8_scalars* scalars_dev, const zs_adamw_q8_tensor* tensors,
                                         int32_t count, int32_t param_dtype, int32_t grad_dtype,
                                         const double* norm_sq_dev, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* ZSHARD_TENSORS_H */
