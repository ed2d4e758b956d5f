"""The orthogonalised momentum step over a model's matrices, on the library's
entry points.

MuonOptimizer steps the matrices of a model (attention and MLP projections,
stacks of experts); TensorOptimizer keeps what is left (embeddings, norm
vectors).  A step is the squared norm over the gradients (if clipping, or asked
for, and not given), then muon_step_matrices, one call per distinct weight
decay.  Nothing here computes; it orders calls.

``state_dict`` / ``load_state_dict`` carry the momentum per tensor (fp32): a
resumed run continues bit for bit.
"""
from __future__ import annotations

from typing import Optional, Sequence, Union

import numpy as np
import torch

from . import matrices as zm
from . import tensors as zt
from .tensor_step import _decays, _given_norm, _refuse_overlap, _written


class MuonOptimizer:
    """Orthogonalised momentum over `params` (contiguous fp32 or bf16 GPU
    matrices of one dtype, or 3-D stacks of them, updated in place).
    param_bf16: for fp32 params, bf16 tensors (or None) that receive their
    re-casts.  weight_decay: one value, or one per tensor.  scale: what
    update_scale takes ("rms", "spectral", a number), or one per tensor.
    max_norm > 0 clips to that global norm; compute_norm=True forms the norm
    without clipping (a step on a non-finite norm changes nothing).  The
    parameters' storages must stay, and every one needs a gradient."""

    def __init__(self, params: Sequence[torch.Tensor], *, lr: float, momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: Union[float, Sequence[float]] = 0.0, ns_steps: int = 5, coefficients=zm.COEFFICIENTS,
                 eps: float = 1e-7, scale="rms", grad_scale: float = 1.0, max_norm: float = 0.0,
                 param_bf16: Optional[Sequence[Optional[torch.Tensor]]] = None, compute_norm: Optional[bool] = None):
        params = [p.detach() if isinstance(p, torch.Tensor) else p for p in params]
        if not params:
            raise ValueError("params: at least one tensor")
        decays = _decays(weight_decay, len(params))
        scales = [scale] * len(params) if isinstance(scale, str) or np.isscalar(scale) else list(scale)
        for name, ts in (("param_bf16", param_bf16), ("scale", scales)):
            if ts is not None and len(ts) != len(params):
                raise ValueError(f"{name}: {len(ts)} values for {len(params)} tensors")
        checked = zt.GradTensors(params)   # the tensors' checks, before anything is allocated
        zm._matrices(params, "params")
        if param_bf16 is not None:
            param_bf16 = [t.detach() if isinstance(t, torch.Tensor) else t for t in param_bf16]
        self.params = params
        self.lr, self.momentum, self.nesterov = lr, momentum, nesterov
        self.ns_steps, self.coefficients, self.eps = ns_steps, coefficients, eps
        self.grad_scale, self.max_norm = grad_scale, max_norm
        self.compute_norm = (max_norm > 0) if compute_norm is None else compute_norm
        self._check_clip(None)
        for decay in decays:
            zm.muon_scalars_bytes(self._hp(decay, 0.0))   # the hyperparameters' checks
        self._lo, self._hi = _written(params, param_bf16)
        self._momentum = [torch.zeros_like(p, dtype=torch.float32) for p in params]
        # one list per distinct decay, in the order of their first tensors
        self._groups = []
        for decay in dict.fromkeys(decays):
            at = [k for k, d in enumerate(decays) if d == decay]
            pick = lambda ts: None if ts is None else [ts[k] for k in at]  # noqa: E731
            # the parameters stand in for the gradients until these are known
            lst = zm.MuonMatrices(pick(params), pick(params), pick(self._momentum), pick(param_bf16), pick(scales))
            self._groups.append((decay, at, lst))
        self._grads: Optional[zt.GradTensors] = None
        dev = params[0].device
        self.norm_sq = torch.zeros(1, dtype=torch.float64, device=dev)
        need = [zm.muon_step_matrices_workspace_bytes(lst) for _, _, lst in self._groups]
        # for gradients of either dtype: a run on another stream never sees it move
        need += [zt._lib().grad_norm_sq_tensors_workspace_bytes(checked.address, checked.count, d) for d in (0, 1)]
        self._workspace = torch.empty(max(need + [256]), dtype=torch.uint8, device=dev)
        self.t = 0

    def bind_grads(self, grads: Sequence[torch.Tensor]) -> None:
        """The gradients of the steps to come, one per parameter, of its shape
        (fp32 or bf16, one dtype): buffers that are refilled in place are bound once."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError("bind_grads: one gradient per parameter")
        lst = zt.GradTensors(grads)
        if any(g.shape != p.shape for g, p in zip(grads, self.params)):
            raise ValueError("bind_grads: a gradient has its parameter's shape")
        _refuse_overlap(lst, self._lo, self._hi)
        for _, at, group in self._groups:
            group.set_grads([grads[k] for k in at])
        self._grads = lst

    def _check_clip(self, norm_sq) -> None:
        if self.max_norm > 0 and not self.compute_norm and norm_sq is None:
            raise ValueError("max_norm > 0 needs the norm: compute_norm")

    def _hp(self, decay: float, extra_norm_sq: float) -> zm.MuonConfig:
        return zm.MuonConfig(lr=self.lr, momentum=self.momentum, nesterov=self.nesterov, weight_decay=decay,
                             ns_steps=self.ns_steps, coefficients=self.coefficients, eps=self.eps,
                             grad_scale=self.grad_scale, max_norm=self.max_norm, extra_norm_sq=extra_norm_sq)

    def step(self, grads: Optional[Sequence[torch.Tensor]] = None, extra_norm_sq: float = 0.0,
             norm_sq: Optional[torch.Tensor] = None) -> None:
        """One step on `grads` (bound first, see bind_grads), or on the bound
        ones.  norm_sq: the squared norm of the scaled gradients of more than
        these tensors, formed already (fp64, device: one norm for a model that
        two optimizers share); extra_norm_sq: the other ranks' share of it."""
        if grads is not None:
            self.bind_grads(grads)
        if self._grads is None:
            raise RuntimeError("step() without gradients")
        self._check_clip(norm_sq)
        configs = [self._hp(decay, extra_norm_sq) for decay, _, _ in self._groups]
        if len(configs) > 1:   # what one call would refuse is refused before another has run
            for hp in configs:
                zm.muon_scalars_bytes(hp)
        norm = norm_sq
        if norm is None and self.compute_norm:
            norm = zt.grad_norm_sq_tensors(self._grads, self.grad_scale, self.norm_sq, self._workspace)
        for hp, (_, _, lst) in zip(configs, self._groups):
            zm.muon_step_matrices(hp, lst, norm_sq=norm, workspace=self._workspace)
        self.t += 1

    def capture(self, extra_norm_sq: float = 0.0, norm_sq: Optional[torch.Tensor] = None) -> "CapturedMuonStep":
        """Record one step on the bound gradients in a HIP graph that replays
        every later step (its scalars are read from device memory; a norm_sq that
        is given, from its tensor).  Capturing changes neither parameters nor
        momentum."""
        return CapturedMuonStep(self, extra_norm_sq, norm_sq)

    def state_dict(self) -> dict:
        return {"step": self.t, "momentum": list(self._momentum)}

    def load_state_dict(self, state: dict) -> None:
        """Take a state_dict's momentum (any device) and step counter."""
        ts, t = state["momentum"], int(state["step"])
        if [tuple(x.shape) for x in ts] != [tuple(p.shape) for p in self.params] or \
                any(x.dtype != torch.float32 for x in ts):
            raise ValueError(f"load_state_dict: momentum must hold {len(self.params)} float32 tensors of the "
                             "parameters' shapes")
        if t < 0:
            raise ValueError("load_state_dict: step must be >= 0")
        for to, src in zip(self._momentum, ts):
            to.copy_(src)
        self.t = t


class CapturedMuonStep:
    """One MuonOptimizer step captured in a HIP graph (MuonOptimizer.capture).
    replay() runs the next step on the gradients that were bound.  The graph has a
    workspace of its own."""

    def __init__(self, opt: MuonOptimizer, extra_norm_sq: float, norm_sq: Optional[torch.Tensor]):
        if opt._grads is None:
            raise RuntimeError("capture() without bound gradients")
        opt._check_clip(norm_sq)
        self.opt, self.extra_norm_sq = opt, extra_norm_sq
        self._norm = _given_norm(norm_sq, "capture")
        self._fixed = self._now()   # in the recorded launches, not in device memory
        # what the graph reads and writes stays this object's, whatever is bound later
        self._grads = opt._grads
        self._lists = [(decay, lst.clone()) for decay, _, lst in opt._groups]
        dev = opt.norm_sq.device
        self._norm_sq = torch.zeros_like(opt.norm_sq)
        self._workspace = torch.empty_like(opt._workspace)
        size = len(self._bytes(0))
        self._host = torch.empty(size * len(self._lists), dtype=torch.uint8, pin_memory=True)
        self._dev = torch.empty(size * len(self._lists), dtype=torch.uint8, device=dev)
        self._parts = self._dev.split(size)
        self._done = torch.cuda.Event()
        self._write()
        # one warm-up run on a side stream, as capture requires, on a norm that is
        # not finite: the step leaves everything as it is
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            self._body(torch.full_like(opt.norm_sq, float("nan")))
        torch.cuda.current_stream(dev).wait_stream(side)
        torch.cuda.synchronize(dev)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._body()

    def _now(self):
        return (self.opt.grad_scale, self.opt.compute_norm, self.opt.ns_steps)

    def _bytes(self, k: int) -> bytes:
        return zm.muon_scalars_bytes(self.opt._hp(self._lists[k][0], self.extra_norm_sq))

    def _write(self) -> None:
        raw = b"".join(self._bytes(k) for k in range(len(self._lists)))
        self._host.numpy()[:] = np.frombuffer(raw, dtype=np.uint8)

    def _body(self, warm_up_norm: Optional[torch.Tensor] = None) -> None:
        opt = self.opt
        norm = self._norm
        if norm is None and opt.compute_norm:
            norm = zt.grad_norm_sq_tensors(self._grads, opt.grad_scale, self._norm_sq, self._workspace)
        norm = norm if warm_up_norm is None else warm_up_norm
        self._dev.copy_(self._host, non_blocking=True)
        for (_, lst), sc in zip(self._lists, self._parts):
            zm.muon_step_matrices_dev(sc, opt.ns_steps, lst, norm_sq=norm, workspace=self._workspace)

    def replay(self) -> None:
        """Run the next step.  Waits for the previous replay to have read the
        pinned scalars before rewriting them.  lr, momentum, nesterov,
        coefficients, eps and max_norm are the optimizer's of now; grad_scale,
        compute_norm and ns_steps must be those of the capture."""
        self.opt._check_clip(self._norm)
        if self._fixed != self._now():
            raise RuntimeError("replay(): grad_scale, compute_norm or ns_steps changed since the capture")
        self._done.synchronize()
        self._write()
        self.graph.replay()
        self._done.record()
        self.opt.t += 1
