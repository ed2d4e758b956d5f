"""The optimizer step over a list of tensors, on the library's entry points.

ShardOptimizer steps one rank's flat shard; TensorOptimizer steps a model as
the list of its parameters (plain data parallelism, tensors kept out of the
flat units, per-parameter sharding).  A step is the squared norm over all
gradients (if clipping, or asked for), then AdamW over the list, one call per
distinct weight decay.  Nothing here computes; it orders calls.

``state_bits=32`` keeps fp32 moments; ``state_bits=8`` keeps them in 8 bits
(2 instead of 8 bytes per element) with unbiased stochastic rounding that
depends on ``seed``, the step and an element's place alone.

``state_dict`` / ``load_state_dict`` carry the step counter and fp32 moments
per tensor, whatever the width: a resumed run continues bit for bit (8-bit
values are exact in fp32 and are stored back exactly), and a run may go on
under the other width.
"""
from __future__ import annotations

from typing import Optional, Sequence, Union

import numpy as np
import torch

from . import _binding as zs
from . import tensors as zt


def _moments_like(params: Sequence[torch.Tensor]) -> list:
    """fp32 zeros for each tensor, views of one buffer.  Each starts at its
    parameter's element offset from a boundary of 256 elements, so that the step
    can put every stream it reads and writes on whole tiles; those of parameters
    that follow one another do so too."""
    buffer = torch.zeros(sum(p.numel() + 256 for p in params) + 256, dtype=torch.float32, device=params[0].device)
    first, views = buffer.data_ptr() // 4, []
    at = 0
    for p in params:
        at += (p.data_ptr() // p.element_size() - first - at) % 256
        views.append(buffer[at:at + p.numel()])
        at += p.numel()
    return views


def _states_for(params: Sequence[torch.Tensor]) -> list:
    """Zeroed 8-bit moments for each tensor, views of one buffer, each on a
    boundary of 1 KiB (what a wave reads of them at once)."""
    sizes = [zt.moments_q8_bytes(p.numel()) for p in params]
    room = [-(-n // 1024) * 1024 for n in sizes]
    buffer = torch.zeros(sum(room) + 1024, dtype=torch.uint8, device=params[0].device)
    at, views = -buffer.data_ptr() % 1024, []
    for n, r in zip(sizes, room):
        views.append(buffer[at:at + n])
        at += r
    return views


def _written(params: Sequence[torch.Tensor], copies) -> tuple:
    """First and past-last addresses of what a step writes of the caller's, in
    ascending order.  The library refuses overlaps inside one call; a step is a
    call per weight decay."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                   for t in [*params, *(copies or [])] if t is not None and t.numel())
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        raise ValueError("params and param_bf16 must not overlap")
    lo, hi = np.array(spans, dtype=np.uint64).reshape(-1, 2).T
    return lo, hi


class TensorOptimizer:
    """AdamW over `params` (contiguous fp32 or bf16 GPU tensors of one dtype,
    updated in place).  param_bf16: for fp32 params, bf16 tensors (or None) that
    receive their re-casts.  weight_decay: one value, or one per tensor.
    max_norm > 0 clips to that global norm; compute_norm=True forms the norm
    without clipping (a step on a non-finite norm changes nothing).  The
    parameters' storages must stay (a parameter moved or resized afterwards is
    not followed), and every one needs a gradient."""

    def __init__(self, params: Sequence[torch.Tensor], *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: Union[float, Sequence[float]] = 0.0, grad_scale: float = 1.0, max_norm: float = 0.0,
                 param_bf16: Optional[Sequence[Optional[torch.Tensor]]] = None, compute_norm: Optional[bool] = None,
                 state_bits: int = 32, seed: int = 0):
        params = [p.detach() if isinstance(p, torch.Tensor) else p for p in params]
        if not params:
            raise ValueError("params: at least one tensor")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        decays = [float(weight_decay)] * len(params) if np.isscalar(weight_decay) else [float(d) for d in weight_decay]
        if len(decays) != len(params):
            raise ValueError(f"weight_decay: {len(decays)} values for {len(params)} tensors")
        if not all(0.0 <= d < float("inf") for d in decays):
            raise ValueError("weight_decay: finite values >= 0")
        if param_bf16 is not None and len(param_bf16) != len(params):
            raise ValueError(f"param_bf16: {len(param_bf16)} tensors for {len(params)}")
        checked = zt.GradTensors(params)   # the tensors' checks, before anything is allocated
        self.params, self.state_bits, self.seed = params, state_bits, zt._seed(seed, "TensorOptimizer")
        self.lr, self.betas, self.eps = lr, betas, eps
        self.grad_scale, self.max_norm = grad_scale, max_norm
        self.compute_norm = (max_norm > 0) if compute_norm is None else compute_norm
        self._check_clip()
        self._lo, self._hi = _written(params, param_bf16)
        if state_bits == 32:
            self._exp_avg, self._exp_avg_sq = _moments_like(params), _moments_like(params)
        else:
            self._states = _states_for(params)
        # one list per distinct decay, in the order of their first tensors
        self._groups = []
        for decay in dict.fromkeys(decays):
            at = [k for k, d in enumerate(decays) if d == decay]
            pick = lambda ts: None if ts is None else [ts[k] for k in at]  # noqa: E731
            # the parameters stand in for the gradients until these are known
            if state_bits == 32:
                lst = zt.AdamWTensors(pick(params), pick(params), pick(self._exp_avg), pick(self._exp_avg_sq),
                                      pick(param_bf16))
            else:
                lst = zt.AdamWQ8Tensors(pick(params), pick(params), pick(self._states), pick(param_bf16))
            self._groups.append((decay, at, lst))
        self._grads: Optional[zt.GradTensors] = None
        dev = params[0].device
        self.norm_sq = torch.zeros(1, dtype=torch.float64, device=dev)
        # for gradients of either dtype: a run on another stream never sees it move
        need = [zt._lib().grad_norm_sq_tensors_workspace_bytes(checked.address, checked.count, dtype)
                for dtype in (zs.ZS_F32, zs.ZS_BF16)]
        self._workspace = torch.empty(max(need + [8]), dtype=torch.uint8, device=dev)
        self.t = 0

    def bind_grads(self, grads: Sequence[torch.Tensor]) -> None:
        """The gradients of the steps to come, one per parameter (fp32 or bf16,
        one dtype): buffers that are refilled in place are bound once.  Binding
        costs the host about 0.7 us a tensor."""
        lst = zt.GradTensors(list(grads))
        if lst.numels != [p.numel() for p in self.params]:
            raise ValueError("bind_grads: one gradient per parameter, of its size")
        # the first buffer that is written and ends after a gradient's start, if any
        at = np.searchsorted(self._hi, lst.array["ptr"][:lst.count], side="right")
        lo = np.append(self._lo, np.uint64(0xFFFFFFFFFFFFFFFF))[at]
        sizes = np.array(lst.numels) * (2 if lst.grad_dtype == zs.ZS_BF16 else 4)
        if ((lo < lst.array["ptr"][:lst.count] + sizes.astype(np.uint64)) & (sizes > 0)).any():
            raise ValueError("bind_grads: a gradient overlaps a parameter or a re-cast")
        for _, at, group in self._groups:
            group._take_grads(lst, at)
        self._grads = lst

    def _check_clip(self) -> None:
        if self.max_norm > 0 and not self.compute_norm:
            raise ValueError("max_norm > 0 needs the norm: compute_norm")

    def _hp(self, decay: float, extra_norm_sq: float, t: int) -> zs.AdamWConfig:
        return zs.AdamWConfig(lr=self.lr, beta1=self.betas[0], beta2=self.betas[1], eps=self.eps, weight_decay=decay,
                              grad_scale=self.grad_scale, max_norm=self.max_norm, extra_norm_sq=extra_norm_sq, step=t)

    def _group_seed(self, k: int) -> int:
        return (self.seed + k) % (1 << 32)

    def step(self, grads: Optional[Sequence[torch.Tensor]] = None, extra_norm_sq: float = 0.0) -> None:
        """One step on `grads` (bound first, see bind_grads), or on the bound
        ones.  extra_norm_sq: the other ranks' share of the squared norm.  The
        step counter advances only once the update is enqueued."""
        if grads is not None:
            self.bind_grads(grads)
        if self._grads is None:
            raise RuntimeError("step() without gradients")
        self._check_clip()
        norm = None
        if self.compute_norm:
            norm = zt.grad_norm_sq_tensors(self._grads, self.grad_scale, self.norm_sq, self._workspace)
        for k, (decay, _, lst) in enumerate(self._groups):
            hp = self._hp(decay, extra_norm_sq, self.t + 1)
            if self.state_bits == 32:
                zt.adamw_step_tensors(hp, lst, norm_sq=norm)
            else:
                zt.adamw_step_tensors_q8(hp, lst, seed=self._group_seed(k), norm_sq=norm)
        self.t += 1

    def capture(self, extra_norm_sq: float = 0.0) -> "CapturedTensorStep":
        """Record one step on the bound gradients in a HIP graph that replays
        every later step (its scalars are read from device memory).  Capturing
        changes neither parameters nor moments."""
        return CapturedTensorStep(self, extra_norm_sq)

    def _moments(self, exp_avg, exp_avg_sq) -> zt.Q8Moments:
        return zt.Q8Moments(self._states, exp_avg, exp_avg_sq, [p.numel() for p in self.params])

    def moments(self):
        """(exp_avg, exp_avg_sq): lists of fp32 tensors; the live ones for 32
        bits, fresh copies of the values for 8."""
        if self.state_bits == 32:
            return self._exp_avg, self._exp_avg_sq
        out = [[torch.empty(p.numel(), dtype=torch.float32, device=p.device) for p in self.params] for _ in range(2)]
        zt.moments_q8_decode(self._moments(*out))
        return out[0], out[1]

    def state_dict(self) -> dict:
        m, v = self.moments()
        return {"step": self.t, "exp_avg": list(m), "exp_avg_sq": list(v)}

    def load_state_dict(self, state: dict) -> None:
        """Take a state_dict's moments (any device) and step counter."""
        numels = [p.numel() for p in self.params]
        for name in ("exp_avg", "exp_avg_sq"):   # every check before the first copy: a refused state changes nothing
            ts = state[name]
            if [t.numel() for t in ts] != numels or any(t.dtype != torch.float32 for t in ts):
                raise ValueError(f"load_state_dict: {name} must hold {len(numels)} float32 tensors of the parameters' sizes")
        t = int(state["step"])
        if t < 0:
            raise ValueError("load_state_dict: step must be >= 0")
        dev = self.norm_sq.device
        if self.state_bits == 32:
            for name, own in (("exp_avg", self._exp_avg), ("exp_avg_sq", self._exp_avg_sq)):
                for to, src in zip(own, state[name]):
                    to.copy_(src.reshape(-1))
        else:
            m, v = ([x.reshape(-1).to(dev).contiguous() for x in state[name]] for name in ("exp_avg", "exp_avg_sq"))
            zt.moments_q8_encode(self._moments(m, v), seed=self.seed)
        self.t = t


class CapturedTensorStep:
    """One TensorOptimizer step captured in a HIP graph (TensorOptimizer.capture).
    replay() runs the next step, t + 1, on the gradients that were bound."""

    def __init__(self, opt: TensorOptimizer, extra_norm_sq: float):
        if opt._grads is None:
            raise RuntimeError("capture() without bound gradients")
        opt._check_clip()
        self.opt, self.extra_norm_sq = opt, extra_norm_sq
        self._fixed = (opt.grad_scale, opt.compute_norm)   # in the recorded launches, not in device memory
        # what the graph reads and writes stays this object's, whatever is bound later
        self._grads = opt._grads
        self._lists = [(decay, lst.clone()) for decay, _, lst in opt._groups]
        dev = opt.norm_sq.device
        size = len(self._bytes(0, 1))
        self._host = torch.empty(size * len(self._lists), dtype=torch.uint8, pin_memory=True)
        self._dev = torch.empty(size * len(self._lists), dtype=torch.uint8, device=dev)
        self._parts = self._dev.split(size)
        self._done = torch.cuda.Event()
        self._write(opt.t + 1)
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

    def _bytes(self, k: int, t: int) -> bytes:
        hp = self.opt._hp(self._lists[k][0], self.extra_norm_sq, t)
        return zs.scalars_bytes(hp) if self.opt.state_bits == 32 else \
            zt.q8_scalars_bytes(hp, self.opt._group_seed(k))

    def _write(self, t: int) -> None:
        raw = b"".join(self._bytes(k, t) for k in range(len(self._lists)))
        self._host.numpy()[:] = np.frombuffer(raw, dtype=np.uint8)

    def _body(self, warm_up_norm: Optional[torch.Tensor] = None) -> None:
        opt = self.opt
        norm = None
        if opt.compute_norm:
            norm = zt.grad_norm_sq_tensors(self._grads, opt.grad_scale, opt.norm_sq, opt._workspace)
        norm = norm if warm_up_norm is None else warm_up_norm
        self._dev.copy_(self._host, non_blocking=True)
        for (_, lst), sc in zip(self._lists, self._parts):
            if opt.state_bits == 32:
                zt.adamw_step_tensors_dev(sc, lst, norm_sq=norm)
            else:
                zt.adamw_step_tensors_q8_dev(sc, lst, norm_sq=norm)

    def replay(self) -> None:
        """Run the next step.  Waits for the previous replay to have read the
        pinned scalars before rewriting them.  lr, betas, eps and max_norm are
        the optimizer's of now; grad_scale and compute_norm must be those of
        the capture (the norm was recorded with them)."""
        self.opt._check_clip()
        if self._fixed != (self.opt.grad_scale, self.opt.compute_norm):
            raise RuntimeError("replay(): grad_scale or compute_norm changed since the capture")
        self._done.synchronize()
        self._write(self.opt.t + 1)
        self.graph.replay()
        self._done.record()
        self.opt.t += 1
