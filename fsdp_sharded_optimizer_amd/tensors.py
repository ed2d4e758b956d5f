"""ctypes binding of the calls over lists of tensors (include/zshard_tensors.h).

A list is marshalled once, into an object that holds its tensors and their
C descriptors (GradTensors, AdamWTensors, AdamWQ8Tensors, Q8Moments), and
passed to every call: a program's parameters and moments stay where they are
from step to step, and a list of some hundred tensors costs more to marshal
than to step.  Nothing is cached behind a call: a gradient that moved is given
anew with ``set_grads``.  A list holds its tensors, but cannot hold a storage
that is replaced or resized under one (``t.data = ...``, ``resize_``): such a
list is marshalled anew before its next call.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Union

import numpy as np
import torch

from . import _binding as zs

Q8_BLOCK = 256   # ZS_Q8_BLOCK: elements that share a scale

# every symbol include/zshard_tensors.h declares
TENSOR_EXPORTS = (
    "grad_norm_sq_tensors_workspace_bytes", "grad_norm_sq_tensors", "adamw_step_tensors", "adamw_step_tensors_dev",
    "moments_q8_bytes", "moments_q8_encode", "moments_q8_decode", "adamw_step_tensors_q8", "adamw_q8_scalars",
    "adamw_step_tensors_q8_dev",
)


def _struct(name: str, pointers: Sequence[str]):
    fields = [(p, ctypes.c_void_p) for p in pointers] + [("numel", ctypes.c_int64)]
    return type(name, (ctypes.Structure,), {"_fields_": fields})


AdamWTensor = _struct("AdamWTensor", ("param", "grad", "exp_avg", "exp_avg_sq", "param_bf16"))
AdamWQ8Tensor = _struct("AdamWQ8Tensor", ("param", "grad", "state_q8", "param_bf16"))
MomentsQ8 = _struct("MomentsQ8", ("exp_avg", "exp_avg_sq", "state_q8"))


class AdamWQ8Scalars(ctypes.Structure):
    """zs_adamw_q8_scalars: one step's binary32 scalars and its key (64 bytes)."""
    _fields_ = [("adamw", zs.AdamWScalars), ("key", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    L = zs.lib()
    if _ready is not L:
        P, I32, U32, I64, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_int64, ctypes.c_double
        HP = ctypes.POINTER(zs.AdamW)
        for name, args, res in (
                ("grad_norm_sq_tensors_workspace_bytes", [P, I32, I32], I64),
                ("grad_norm_sq_tensors", [P, I32, I32, D, P, P, I64, P], I32),
                ("adamw_step_tensors", [HP, P, I32, I32, I32, P, P], I32),
                ("adamw_step_tensors_dev", [P, P, I32, I32, I32, P, P], I32),
                ("moments_q8_bytes", [I64], I64),
                ("moments_q8_encode", [P, I32, I32, U32, P], I32),
                ("moments_q8_decode", [P, I32, I32, P], I32),
                ("adamw_step_tensors_q8", [HP, U32, P, I32, I32, I32, P, P], I32),
                ("adamw_q8_scalars", [HP, U32, ctypes.POINTER(AdamWQ8Scalars)], I32),
                ("adamw_step_tensors_q8_dev", [P, P, I32, I32, I32, P, P], I32)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _ready = L
    return L


# ---------------------------------------------------------------------------
# lists
# ---------------------------------------------------------------------------

def _pointers(ts: Sequence[Optional[torch.Tensor]], name: str, numels: Sequence[int], dtypes, optional: bool = False):
    """Device pointers of one kind of tensor, and their common dtype (None
    where every tensor is None).  One pass with the checks of zs._dev, which is
    called only to say what is wrong: a list is some hundred tensors."""
    if len(ts) != len(numels):
        raise ValueError(f"{name}: {len(ts)} tensors, the list has {len(numels)}")
    kind, out, device = None, [], torch.cuda.current_device() if torch.cuda.is_available() else -1
    for k, (t, n) in enumerate(zip(ts, numels)):
        if t is None and optional:
            out.append(0)
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{k}]: expected a torch.Tensor")
        if not t.is_cuda or t.get_device() != device or not t.is_contiguous():
            zs._dev(t, f"{name}[{k}]")
        if kind is None:
            kind = t.dtype
        if t.dtype != kind or kind not in dtypes:
            raise TypeError(f"{name}[{k}]: {t.dtype}; one of {', '.join(map(str, dtypes))}, the same for all")
        if t.numel() != n:
            raise ValueError(f"{name}[{k}]: size mismatch")
        out.append(t.data_ptr())
    return out, kind


class _List:
    """A marshalled list: `array` (count descriptors), and the tensors it
    points into, kept alive."""

    def __init__(self, struct, numels: Sequence[int], device):
        self.count = len(numels)
        self.numels = list(numels)
        self.array = np.zeros(max(self.count, 1), dtype=np.dtype(struct))
        self.address = self.array.ctypes.data
        self.array["numel"][:self.count] = self.numels
        self.device = device
        self.tensors = {}

    def _set(self, field: str, ts, pointers) -> None:
        self.array[field][:self.count] = pointers
        self.tensors[field] = list(ts) if ts is not None else None

    def clone(self) -> "_List":
        """The list as it is now (the same tensors): later set_grads on either
        leave the other alone."""
        out = object.__new__(type(self))
        out.__dict__.update(self.__dict__)
        out.array = self.array.copy()
        out.address = out.array.ctypes.data
        out.tensors = dict(self.tensors)
        return out

    def check(self, fn: str) -> None:
        if self.count and self.device.index != torch.cuda.current_device():
            raise ValueError(f"{fn}: list on {self.device}, but the current device is "
                             f"cuda:{torch.cuda.current_device()}")


_FLOATS = (torch.float32, torch.bfloat16)


def _numels(ts: Sequence[torch.Tensor], name: str):
    for k, t in enumerate(ts):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{k}]: expected a torch.Tensor")
    return [t.numel() for t in ts], (ts[0].device if len(ts) else None)


class GradTensors(_List):
    """Gradients (fp32 or bf16, one dtype) for grad_norm_sq_tensors."""

    def __init__(self, grads: Sequence[torch.Tensor]):
        grads = list(grads)
        numels, device = _numels(grads, "grads")
        super().__init__(zs.Tensor, numels, device)
        self.set_grads(grads)

    def set_grads(self, grads: Sequence[torch.Tensor]) -> None:
        """Other tensors of the same sizes."""
        pointers, dtype = _pointers(grads, "grads", self.numels, _FLOATS)
        self._set("ptr", grads, pointers)
        self.grad_dtype = zs.ZS_BF16 if dtype == torch.bfloat16 else zs.ZS_F32


class _StepList(_List):
    def _params(self, params, param_bf16) -> None:
        pointers, dtype = _pointers(params, "params", self.numels, _FLOATS)
        self._set("param", params, pointers)
        self.param_dtype = zs.ZS_BF16 if dtype == torch.bfloat16 else zs.ZS_F32
        if param_bf16 is not None:
            if dtype == torch.bfloat16 and any(t is not None for t in param_bf16):
                raise ValueError("param_bf16: a re-cast of fp32 parameters; these are bf16")
            pointers, _ = _pointers(param_bf16, "param_bf16", self.numels, (torch.bfloat16,), optional=True)
            self._set("param_bf16", param_bf16, pointers)

    def set_grads(self, grads: Union["GradTensors", Sequence[torch.Tensor]]) -> None:
        """Other gradients of the same sizes (fp32 or bf16, one dtype)."""
        if not isinstance(grads, GradTensors):
            grads = GradTensors(grads)
        self._take_grads(grads, range(grads.count))

    def _take_grads(self, grads: "GradTensors", at: Sequence[int]) -> None:
        """The tensors `at` of a checked list of gradients."""
        if grads.device != self.device and grads.count:   # it may have been marshalled while another GPU was current
            raise ValueError(f"grads on {grads.device}, the list on {self.device}")
        at = np.fromiter(at, dtype=np.int64)
        if [grads.numels[k] for k in at] != self.numels:
            raise ValueError("grads: one per tensor of the list, of its size")
        self._set("grad", [grads.tensors["ptr"][k] for k in at], grads.array["ptr"][at])
        self.grad_dtype = grads.grad_dtype


class AdamWTensors(_StepList):
    """The tensors of adamw_step_tensors: params (fp32 or bf16), grads (fp32 or
    bf16), exp_avg and exp_avg_sq (fp32), and for fp32 params their bf16
    re-casts (a list with None where a tensor has none, or None)."""

    def __init__(self, params, grads, exp_avg, exp_avg_sq, param_bf16=None):
        numels, device = _numels(params, "params")
        super().__init__(AdamWTensor, numels, device)
        self._params(params, param_bf16)
        self.set_grads(grads)
        for name, ts in (("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
            self._set(name, ts, _pointers(ts, name, self.numels, (torch.float32,))[0])


def _states(ts, numels):
    """Device pointers of 8-bit moments, large enough for the numels."""
    if len(ts) != len(numels):
        raise ValueError(f"states: {len(ts)} tensors, the list has {len(numels)}")
    for k, t in enumerate(ts):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"states[{k}]: expected a torch.Tensor")
    pointers, _ = _pointers(ts, "states", [t.numel() for t in ts], (torch.uint8,))
    for k, (t, n) in enumerate(zip(ts, numels)):
        if t.numel() < moments_q8_bytes(n):
            raise ValueError(f"states[{k}]: holds {t.numel()} bytes, the 8-bit moments of {n} elements need "
                             f"{moments_q8_bytes(n)}")
    return pointers


class AdamWQ8Tensors(_StepList):
    """The tensors of adamw_step_tensors_q8: as AdamWTensors, with each
    tensor's moments in one uint8 tensor of moments_q8_bytes(numel) bytes
    (zeros: a fresh optimizer)."""

    def __init__(self, params, grads, states, param_bf16=None):
        numels, device = _numels(params, "params")
        super().__init__(AdamWQ8Tensor, numels, device)
        self._params(params, param_bf16)
        self.set_grads(grads)
        self._set("state_q8", states, _states(states, self.numels))


class Q8Moments(_List):
    """The tensors of moments_q8_encode and moments_q8_decode: 8-bit moments and
    their exp_avg and exp_avg_sq (fp32 or bf16, one dtype; a list may be None,
    or hold None).  numels: where both lists are None."""

    def __init__(self, states, exp_avg, exp_avg_sq, numels: Optional[Sequence[int]] = None):
        count = len(states)
        lists = [[None] * count if ts is None else list(ts) for ts in (exp_avg, exp_avg_sq)]
        for name, ts in zip(("exp_avg", "exp_avg_sq"), lists):
            if len(ts) != count:
                raise ValueError(f"{name}: {len(ts)} tensors, the list has {count}")
        if numels is None:
            numels = []
            for k, pair in enumerate(zip(*lists)):
                t = next((t for t in pair if t is not None), None)
                if t is None:
                    raise ValueError(f"tensor {k} has neither moment: give numels")
                numels.append(t.numel())
        pointers = _states(states, numels)
        super().__init__(MomentsQ8, numels, states[0].device if count else None)
        self._set("state_q8", states, pointers)
        kinds = []
        for name, ts in zip(("exp_avg", "exp_avg_sq"), lists):
            pointers, kind = _pointers(ts, name, self.numels, _FLOATS, optional=True)
            self._set(name, ts, pointers)
            kinds += [kind] if kind is not None else []
        if len(set(kinds)) > 1:
            raise TypeError("exp_avg and exp_avg_sq must share one dtype")
        self.dtype = zs.ZS_BF16 if kinds and kinds[0] == torch.bfloat16 else zs.ZS_F32


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def _grad_list(grads) -> GradTensors:
    return grads if isinstance(grads, GradTensors) else GradTensors(list(grads))


def grad_norm_sq_tensors_workspace_bytes(grads: Union[GradTensors, Sequence[torch.Tensor]]) -> int:
    grads = _grad_list(grads)
    return int(_lib().grad_norm_sq_tensors_workspace_bytes(grads.address, grads.count, grads.grad_dtype))


def grad_norm_sq_tensors(grads: Union[GradTensors, Sequence[torch.Tensor]], grad_scale: float, out: torch.Tensor,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[0] (fp64, device) = sum over the tensors of (fl32(widen(grad) * scale))^2 in binary64."""
    grads = _grad_list(grads)
    grads.check("grad_norm_sq_tensors")
    if out.dtype != torch.float64 or out.numel() < 1:
        raise TypeError("grad_norm_sq_tensors: out must hold one float64")
    if workspace is None:
        # of the stream it is used on: freed at return, it is next used in that stream's order
        with torch.cuda.stream(stream):
            workspace = torch.empty(max(grad_norm_sq_tensors_workspace_bytes(grads), 8), dtype=torch.uint8,
                                    device=out.device)
    zs._check("grad_norm_sq_tensors", _lib().grad_norm_sq_tensors(
        grads.address, grads.count, grads.grad_dtype, float(grad_scale), zs._dev(out, "out"),
        zs._dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), zs._stream(stream)))
    return out


def adamw_step_tensors(hp: zs.AdamWConfig, tensors: AdamWTensors, norm_sq: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """AdamW on every tensor of the list (in place), one clip coefficient for all."""
    tensors.check("adamw_step_tensors")
    c = hp.c_struct()
    zs._check("adamw_step_tensors", _lib().adamw_step_tensors(
        ctypes.byref(c), tensors.address, tensors.count, tensors.param_dtype, tensors.grad_dtype,
        zs._norm(norm_sq, "adamw_step_tensors"), zs._stream(stream)))


def _scalars_dev(t: torch.Tensor, struct, fn: str) -> int:
    if t.dtype != torch.uint8 or t.numel() < ctypes.sizeof(struct):
        raise TypeError(f"{fn}: scalars_dev must be a uint8 tensor of at least {ctypes.sizeof(struct)} bytes")
    return zs._dev(t, "scalars_dev")


def adamw_step_tensors_dev(scalars_dev: torch.Tensor, tensors: AdamWTensors, norm_sq: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """adamw_step_tensors with its scalars read from device memory when the
    kernels run (scalars_dev: uint8 GPU tensor holding scalars_bytes(hp))."""
    tensors.check("adamw_step_tensors_dev")
    zs._check("adamw_step_tensors_dev", _lib().adamw_step_tensors_dev(
        _scalars_dev(scalars_dev, zs.AdamWScalars, "adamw_step_tensors_dev"), tensors.address, tensors.count,
        tensors.param_dtype, tensors.grad_dtype, zs._norm(norm_sq, "adamw_step_tensors_dev"), zs._stream(stream)))


def moments_q8_bytes(n: int) -> int:
    """Bytes of the 8-bit moments of n elements (host only)."""
    out = int(_lib().moments_q8_bytes(int(n)))
    if out < 0:
        raise ValueError(f"moments_q8_bytes: invalid element count {n}")
    return out


def _seed(seed: int, fn: str) -> int:
    if not 0 <= int(seed) < 1 << 32:
        raise ValueError(f"{fn}: seed must fit 32 bits")
    return int(seed)


def moments_q8_encode(moments: Q8Moments, seed: int = 0, stream=None) -> None:
    """exp_avg and exp_avg_sq of every tensor (None: zeros) into its 8-bit state."""
    moments.check("moments_q8_encode")
    zs._check("moments_q8_encode", _lib().moments_q8_encode(
        moments.address, moments.count, moments.dtype, _seed(seed, "moments_q8_encode"), zs._stream(stream)))


def moments_q8_decode(moments: Q8Moments, stream=None) -> None:
    """The values of every tensor's 8-bit state into exp_avg and exp_avg_sq
    (None: skipped); bf16 holds them exactly from 2^-130 up."""
    moments.check("moments_q8_decode")
    zs._check("moments_q8_decode", _lib().moments_q8_decode(
        moments.address, moments.count, moments.dtype, zs._stream(stream)))


def adamw_step_tensors_q8(hp: zs.AdamWConfig, tensors: AdamWQ8Tensors, seed: int = 0,
                          norm_sq: Optional[torch.Tensor] = None, stream=None) -> None:
    """adamw_step_tensors on 8-bit moments; the stochastic rounding of what is
    stored depends on seed, hp.step, a tensor's place in the list and the
    element's place in it alone."""
    tensors.check("adamw_step_tensors_q8")
    c = hp.c_struct()
    zs._check("adamw_step_tensors_q8", _lib().adamw_step_tensors_q8(
        ctypes.byref(c), _seed(seed, "adamw_step_tensors_q8"), tensors.address, tensors.count, tensors.param_dtype,
        tensors.grad_dtype, zs._norm(norm_sq, "adamw_step_tensors_q8"), zs._stream(stream)))


def q8_scalars_bytes(hp: zs.AdamWConfig, seed: int = 0) -> bytes:
    """adamw_q8_scalars(hp, seed) as the bytes adamw_step_tensors_q8_dev reads."""
    out = AdamWQ8Scalars()
    c = hp.c_struct()
    zs._check("adamw_q8_scalars", _lib().adamw_q8_scalars(ctypes.byref(c), _seed(seed, "adamw_q8_scalars"),
                                                          ctypes.byref(out)))
    return bytes(out)


def adamw_step_tensors_q8_dev(scalars_dev: torch.Tensor, tensors: AdamWQ8Tensors,
                              norm_sq: Optional[torch.Tensor] = None, stream=None) -> None:
    """adamw_step_tensors_q8 with its scalars read from device memory when the
    kernels run (scalars_dev: uint8 GPU tensor holding q8_scalars_bytes)."""
    tensors.check("adamw_step_tensors_q8_dev")
    zs._check("adamw_step_tensors_q8_dev", _lib().adamw_step_tensors_q8_dev(
        _scalars_dev(scalars_dev, AdamWQ8Scalars, "adamw_step_tensors_q8_dev"), tensors.address, tensors.count,
        tensors.param_dtype, tensors.grad_dtype, zs._norm(norm_sq, "adamw_step_tensors_q8_dev"),
        zs._stream(stream)))
