"""MI355X-native per-rank ZeRO/FSDP optimizer step (libzshard).

The Python names mirror the C ABI in include/zshard.h:

    zero_shard_range(total, world, rank) -> (chunk, start, end, padded_total)
    flat_pack(src_tensors, flat, padded_total=None)
    flat_unpack(flat, dst_tensors)
    grad_accum(acc, grad, overwrite)
    grad_reduce_chunks(acc, chunks, overwrite)
    grad_reduce_chunks_norm_sq(acc, chunks, overwrite, grad_scale, out, workspace=None)
    grad_accum_norm_sq(acc, grad, overwrite, grad_scale, out, workspace=None)
    grad_accum_norm_sq_noalloc(acc, grad, overwrite, grad_scale, out)   partials in a static device scratch
    grad_norm_sq(grad, grad_scale, out, workspace=None)
    grad_sum_norm_sq(acc, grad, overwrite, grad_scale, out, workspace=None)   grad_accum_norm_sq's norm, no store
    adamw_step(hp, master, exp_avg, exp_avg_sq, grad, param_bf16=None, norm_sq=None)
    adamw_scalars(hp) / scalars_bytes(hp)       the step's binary32 scalars, on the host
    adamw_step_dev(scalars_dev, master, exp_avg, exp_avg_sq, grad, param_bf16=None, norm_sq=None)
    adamw_step_sum(hp, master, exp_avg, exp_avg_sq, acc, grad, param_bf16=None, norm_sq=None)
                                                the step on fl(acc + widen(grad)), the sum not stored
    adamw_step_sum_dev(scalars_dev, master, exp_avg, exp_avg_sq, acc, grad, param_bf16=None, norm_sq=None)
    adamw_step_no_master(hp, param_bf16, exp_avg, exp_avg_sq, grad, norm_sq=None)
    adam_update(hp, exp_avg, exp_avg_sq, grad, update, norm_sq=None)
    flat_apply_update(update, dst_tensors)
    state_tiled_numel(n)                        floats of the tiled optimizer state
    state_tile(master, exp_avg, exp_avg_sq, state, n=None)     split -> tiled (None sources: zeros)
    state_untile(state, master, exp_avg, exp_avg_sq, n=None)   tiled -> split (None: skipped)
    adamw_step_tiled(hp, state, grad, param_bf16=None, norm_sq=None)
    adamw_step_tiled_dev(scalars_dev, state, grad, param_bf16=None, norm_sq=None)
    adamw_step_tiled_sum(hp, state, acc, grad, param_bf16=None, norm_sq=None)   gradient fl(acc + widen(grad))
    adamw_step_tiled_sum_dev(scalars_dev, state, acc, grad, param_bf16=None, norm_sq=None)
    moments_tiled_numel(n) / moments_tile(exp_avg, exp_avg_sq, moments, n=None) / moments_untile(...)
    adam_update_tiled(hp, moments, grad, update, norm_sq=None)
    adamw_step_no_master_tiled(hp, param_bf16, moments, grad, norm_sq=None)

Over lists of tensors (include/zshard_tensors.h), each list marshalled once:

    GradTensors(grads) / AdamWTensors(params, grads, exp_avg, exp_avg_sq, param_bf16=None)
    AdamWQ8Tensors(params, grads, states, param_bf16=None) / Q8Moments(states, exp_avg, exp_avg_sq)
    grad_norm_sq_tensors(grads, grad_scale, out, workspace=None)
    adamw_step_tensors(hp, tensors, norm_sq=None)               fp32 moments; _dev: scalars in device memory
    adamw_step_tensors_q8(hp, tensors, seed=0, norm_sq=None)    8-bit moments; _dev: q8_scalars_bytes(hp, seed)
    moments_q8_bytes(n) / moments_q8_encode(moments, seed=0) / moments_q8_decode(moments)
    MixedTensors(tensors)                                       fp32 and bf16 tensors in one list
    grad_norms_sq_tensors(grads, grad_scale, out, norms=None, workspace=None)   the norm of all, and of each
    grad_clip_tensors(grads, out=None, grad_scale=1.0, max_norm=0.0, norm_sq=None)   scaled, clipped gradients

Over lists of matrices (include/zshard_matrices.h):

    ProductMatrices(a, b, d, c=None) / GramMatrices(a, d, c=None, transposed=None) / OrthogonalizeMatrices(inputs, outputs)
    MuonMatrices(params, grads, momenta, param_bf16=None, scale="rms")
    product_add_matrices(products, alpha=1.0, beta=1.0, workspace=None)         d = alpha op(a) op(b) + beta c
    gram_add_matrices(grams, alpha=1.0, beta=1.0, workspace=None)               d = alpha a a^T + beta c
    orthogonalize_matrices(matrices, steps=5, coefficients=..., eps=1e-7, workspace=None)
    muon_step_matrices(hp, matrices, norm_sq=None, workspace=None)   _dev: muon_scalars_bytes(hp) in device memory

TensorOptimizer(params, lr=..., state_bits=32 or 8) orders the calls over
tensors and MuonOptimizer(matrices, lr=...) those over matrices, as
ShardOptimizer does the calls over a flat shard.

DeviceArena(nbytes, device) holds one physically contiguous block of device
memory and hands out 2 MiB-aligned views of it (ShardOptimizer(arena=...)).

All device work runs in the library's gfx950 HIP kernels on the current
torch stream; torch supplies device memory and the stream only.
"""
from ._binding import (  # noqa: F401
    EXPORTS,
    LIB_PATH,
    NOALLOC_MAX_ELEMS,
    STATE_TILE,
    AdamWConfig,
    ZShardError,
    AdamWScalars,
    adam_update,
    adam_update_tiled,
    adamw_scalars,
    adamw_step,
    adamw_step_dev,
    adamw_step_no_master,
    adamw_step_no_master_tiled,
    adamw_step_sum,
    adamw_step_sum_dev,
    adamw_step_tiled,
    adamw_step_tiled_dev,
    adamw_step_tiled_sum,
    adamw_step_tiled_sum_dev,
    flat_apply_update,
    flat_pack,
    flat_unpack,
    grad_accum,
    grad_accum_norm_sq,
    grad_accum_norm_sq_noalloc,
    grad_accum_norm_sq_workspace_bytes,
    grad_reduce_chunks,
    grad_reduce_chunks_norm_sq,
    grad_reduce_chunks_norm_sq_workspace_bytes,
    grad_norm_sq,
    grad_norm_sq_workspace_bytes,
    grad_sum_norm_sq,
    lib,
    moments_tile,
    moments_tiled_numel,
    moments_untile,
    scalars_bytes,
    state_tile,
    state_tiled_numel,
    state_untile,
    zero_shard_range,
)
from .arena import DeviceArena  # noqa: F401
from .matrices import (  # noqa: F401
    MATRIX_EXPORTS,
    GramMatrices,
    MuonConfig,
    MuonMatrices,
    OrthogonalizeMatrices,
    ProductMatrices,
    gram_add_matrices,
    gram_add_matrices_workspace_bytes,
    muon_scalars_bytes,
    muon_step_matrices,
    muon_step_matrices_dev,
    muon_step_matrices_workspace_bytes,
    orthogonalize_matrices,
    orthogonalize_matrices_workspace_bytes,
    product_add_matrices,
    product_add_matrices_workspace_bytes,
    update_scale,
)
from .muon_step import MuonOptimizer  # noqa: F401
from .step import ShardOptimizer  # noqa: F401
from .tensor_step import TensorOptimizer  # noqa: F401
from .tensors import (  # noqa: F401
    Q8_BLOCK,
    TENSOR_EXPORTS,
    AdamWQ8Scalars,
    AdamWQ8Tensors,
    AdamWTensors,
    GradTensors,
    MixedTensors,
    Q8Moments,
    adamw_step_tensors,
    adamw_step_tensors_dev,
    adamw_step_tensors_q8,
    adamw_step_tensors_q8_dev,
    grad_clip_tensors,
    grad_norm_sq_tensors,
    grad_norm_sq_tensors_workspace_bytes,
    grad_norms_sq_tensors,
    grad_norms_sq_tensors_workspace_bytes,
    moments_q8_bytes,
    moments_q8_decode,
    moments_q8_encode,
    q8_scalars_bytes,
)
