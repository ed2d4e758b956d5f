/*
 * zshard_matrices.h — the optimizer step over a model's matrices (part of
 * libzshard.so; the conventions, types and error codes are zshard.h's): products
 * with a scaled residual, orthogonalisation by Newton-Schulz steps, and the
 * orthogonalised momentum update (Muon) that they make up.
 *
 * Every call takes a host list of device matrices, read during the call only,
 * as the calls of zshard_tensors.h do: tables of it travel in the kernel
 * arguments, nothing is allocated on the device, copied to it or kept, no call
 * blocks, and every call can be captured into a HIP graph as is.  Two calls
 * that may run at the same time (on two streams, or as parts of two graphs)
 * need a workspace each.
 *
 * For every call: count >= 0 and the list not NULL with count > 0.  A matrix is
 * row-major and contiguous; its sides are 0 to ZS_MATRIX_MAX_SIDE and it has
 * fewer than 2^31 elements; one without elements is skipped (its pointers are
 * not looked at).  fp32 pointers are 4-byte and bf16 pointers 2-byte aligned;
 * views at any element offset are fine.  A buffer that is written (a workspace
 * among them) must not overlap any other buffer of the call (ZS_EOVERLAP);
 * buffers that are only read may overlap one another.  The workspace is device
 * memory, 256-byte aligned, at least the bytes that the call's
 * *_workspace_bytes function (host only; -1 for an invalid list) gives for the
 * same list: scratch, owned by the caller until the stream has passed the call.
 */
#ifndef ZSHARD_MATRICES_H
#define ZSHARD_MATRICES_H

#include "zshard.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZS_MATRIX_MAX_SIDE 1048576

/* One product of product_add_matrices. */
typedef struct {
    const void* a;   /* m x k (ZS_TRANSPOSE_A: k x m), of in_dtype, read */
    const void* b;   /* k x n (ZS_TRANSPOSE_B: n x k), of in_dtype, read */
    const void* c;   /* m x n, of c_dtype, read; or NULL */
    void* d;         /* m x n, of d_dtype, written; may be c itself where the dtypes are the same */
    int64_t m, n, k;
} zs_product;

#define ZS_TRANSPOSE_A 1
#define ZS_TRANSPOSE_B 2

/*
 * product_add_matrices — d = alpha * op(a) * op(b) + beta * c for every entry of
 * a list (a preconditioner applied to gradients, with their residual).
 * bf16 inputs: products exact, summed in binary32; alpha, beta and the sum in
 * binary32 (finite there), one rounding to d_dtype.  fp32 inputs are split into two bf16
 * values each (16 significant bits) and three of their four products formed:
 * within 3 * 2^-16 of |a||b| per product (3e-6 of the result in the norm, as
 * measured); an input that is not finite makes what it enters NaN.  c is not
 * read where it is NULL or beta is 0.  k = 0: d = beta * c.
 * in_dtype, c_dtype, d_dtype: ZS_F32 or ZS_BF16; flags: ZS_TRANSPOSE_*.
 * No workspace is needed for bf16 inputs with every k a multiple of 64, no
 * ZS_TRANSPOSE_A, every n a multiple of 8 (or ZS_TRANSPOSE_B), and a and b on
 * 16-byte boundaries (0 bytes then); other inputs are copied into it first.
 * Errors: ZS_EINVAL, ZS_EWORKSPACE, ZS_EOVERLAP, ZS_EHIP.
 */
ZS_API int64_t product_add_matrices_workspace_bytes(const zs_product* list, int32_t count, int32_t in_dtype,
                                                    int32_t flags);
ZS_API int32_t product_add_matrices(const zs_product* list, int32_t count, int32_t in_dtype, int32_t c_dtype,
                                    int32_t d_dtype, int32_t flags, double alpha, double beta, void* workspace,
                                    int64_t workspace_bytes, void* hip_stream);

/* One product of gram_add_matrices. */
typedef struct {
    const void* a;       /* rows x cols, of in_dtype, read */
    const void* c;       /* a symmetric matrix of d's size, of d_dtype, read; or NULL */
    void* d;             /* rows x rows (transposed: cols x cols), of d_dtype, written; may be c itself */
    int64_t rows, cols;
    int32_t transposed;  /* 0: a a^T; 1: a^T a */
    int32_t reserved;    /* 0 */
} zs_gram;

/*
 * gram_add_matrices — d = alpha * a * a^T + beta * c (transposed: a^T * a) for every
 * entry of a list: the running statistics of matrix preconditioners.  As
 * product_add_matrices, but only the tiles on and below the diagonal are formed
 * and the others mirror them: of c only the tiles on and below the diagonal are
 * read, and d is symmetric, bit for bit, where c is.
 */
ZS_API int64_t gram_add_matrices_workspace_bytes(const zs_gram* list, int32_t count, int32_t in_dtype);
ZS_API int32_t gram_add_matrices(const zs_gram* list, int32_t count, int32_t in_dtype, int32_t d_dtype, double alpha,
                                 double beta, void* workspace, int64_t workspace_bytes, void* hip_stream);

/* One matrix of orthogonalize_matrices. */
typedef struct {
    const void* in;      /* rows x cols, of in_dtype, read */
    uint16_t* out;       /* rows x cols, bf16, written */
    int64_t rows, cols;
} zs_orthogonal;

/*
 * orthogonalize_matrices — every matrix of a list with its singular values driven
 * towards 1 (its orthogonal polar factor, nearly):
 *   X = in / max(|in|_F, eps);  `steps` times  X <- a X + (b S + c S^2) X,
 * S = X X^T on the short side (a tall matrix: X <- a X + X (b S + c S^2), S = X^T X).
 * |in|_F is formed in binary64.  X is held scaled by 2^8 as a pair of fp16 values
 * (22 significant bits down to 2^-33, 2^-44 below: a matrix whose norm is 2^-20
 * eps or less), S and b S + c S^2 as one fp16 value each, so scaled; the products
 * take the pair's first value, sums are binary32, and a X the whole pair.  What the
 * linear term amplifies (small singular values, about a^steps times) carries no
 * fp16 rounding therefore: results are within 4e-3 of the formula (relative, in
 * the Frobenius norm; 3e-4 to 2e-3 as measured) for matrices of any rank with the
 * usual coefficients (3.4445, -4.775, 2.0315) and 5 steps, and their rounding to
 * bf16 (2^-8 of a value at most, 1.7e-3 in the norm) comes on top.  Where the
 * short side is 64 or less nothing is held in fp16 alone (the polynomials of S are
 * formed in binary32, of at most 5 steps at a time, and applied to the pair): 1e-6 to
 * 4e-4.  More steps multiply what the first ones were off by as they multiply the
 * matrix: singular values below 2^-22 of the largest are what roundings left there, and
 * grow by a each step until the polynomial holds them.
 * A zero matrix gives zeros, one with a value that is not finite NaN.  steps: 1 to
 * ZS_NS_MAX_STEPS; |a|, |b|, |c| at most 32 and such that X, S and b S + c S^2 stay
 * bounded (fp16 ends at 255 times the scale); eps: at least 1e-30.
 */
#define ZS_NS_MAX_STEPS 32
ZS_API int64_t orthogonalize_matrices_workspace_bytes(const zs_orthogonal* list, int32_t count);
ZS_API int32_t orthogonalize_matrices(const zs_orthogonal* list, int32_t count, int32_t in_dtype, int32_t steps, double a,
                                      double b, double c, double eps, void* workspace, int64_t workspace_bytes,
                                      void* hip_stream);

/* Hyperparameters of one orthogonalised momentum step; lr, lr * weight_decay and
 * grad_scale finite in binary32, grad_scale not 0 there either. */
typedef struct {
    double lr;              /* >= 0 */
    double momentum;        /* [0, 1), in binary32 too */
    double weight_decay;    /* >= 0, decoupled */
    double a, b, c;         /* coefficients of a Newton-Schulz step, as above */
    double eps;             /* >= 1e-30: floor of the Frobenius norm */
    double grad_scale;      /* > 0 */
    double max_norm;        /* > 0: clip to this global norm (needs norm_sq_dev); <= 0: none */
    double extra_norm_sq;   /* >= 0: other ranks' share of the squared norm */
    int32_t nesterov;       /* 0 or 1 */
    int32_t ns_steps;       /* 1 to ZS_NS_MAX_STEPS */
} zs_muon;

/* One matrix of muon_step_matrices. */
typedef struct {
    void* param;            /* rows x cols, of param_dtype, read-write */
    const void* grad;       /* rows x cols, of grad_dtype, read */
    float* momentum;        /* rows x cols, fp32, read-write */
    uint16_t* param_bf16;   /* bf16 re-cast of an fp32 param, written; or NULL */
    int64_t rows, cols;
    double scale;           /* of lr for this matrix, finite; 0.2 sqrt(max(rows, cols)) gives the update AdamW's usual RMS */
} zs_muon_matrix;

/*
 * muon_step_matrices — the orthogonalised momentum update of every matrix of a
 * list.  In binary32, one rounding per operation:
 *   g = widen(grad) * grad_scale * coef     (coef: adamw_step's clip coefficient; 1 without norm_sq_dev)
 *   m = fl(momentum * m) + fl((1 - momentum) * g)
 *   u = nesterov ? fl(momentum * m) + fl((1 - momentum) * g) : m
 *   O = u orthogonalised as by orthogonalize_matrices, kept in binary32
 *   p = fl(p * (1 - lr * weight_decay)) - fl(fl(lr * scale) * O), rounded to param_dtype; its bf16 re-cast
 * A norm that is not finite leaves every matrix and its momentum unchanged.
 * max_norm > 0 without norm_sq_dev clips nothing, as in adamw_step.
 * Errors: ZS_EINVAL, ZS_EWORKSPACE, ZS_EOVERLAP, ZS_EHIP (a list takes many
 * launches: a failed one leaves the earlier ones enqueued).
 */
ZS_API int64_t muon_step_matrices_workspace_bytes(const zs_muon_matrix* list, int32_t count);
ZS_API int32_t muon_step_matrices(const zs_muon* hp, const zs_muon_matrix* list, int32_t count, int32_t param_dtype,
                                  int32_t grad_dtype, const double* norm_sq_dev, void* workspace,
                                  int64_t workspace_bytes, void* hip_stream);

/* A step's scalars as the kernels take them (64 bytes: 8 floats, 2 words, 3 doubles). */
typedef struct {
    float momentum, one_minus_momentum, decay, lr;
    float a, b, c;
    float grad_scale;
    int32_t nesterov, clip;
    double eps;
    double max_norm, extra_norm_sq;
} zs_muon_scalars;

/* The scalars muon_step_matrices forms from hp, on the host. */
ZS_API int32_t muon_scalars(const zs_muon* hp, zs_muon_scalars* out);

/* muon_step_matrices with its scalars read from device memory when the kernels
 * run (8-byte aligned, must not overlap a written buffer): one captured graph
 * replays every step.  The number of Newton-Schulz steps is the launches' and
 * therefore an argument.  The coefficients are not the launches': matrices of a short side
 * up to 64 take longer with |a| above 3.48, and come out the same to rounding. */
ZS_API int32_t muon_step_matrices_dev(const zs_muon_scalars* scalars_dev, int32_t ns_steps, const zs_muon_matrix* list,
                                      int32_t count, int32_t param_dtype, int32_t grad_dtype, const double* norm_sq_dev,
                                      void* workspace, int64_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* ZSHARD_MATRICES_H */
