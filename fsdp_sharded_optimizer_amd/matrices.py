"""ctypes binding of the calls over lists of matrices (include/zshard_matrices.h).

As with the lists of tensors, a list is marshalled once into an object that
holds its matrices and their C descriptors (ProductMatrices, GramMatrices,
OrthogonalizeMatrices, MuonMatrices) and passed to every call.  A matrix is a
contiguous 2-D GPU tensor; a 3-D one is a stack of them (experts' weights).
Each call's workspace comes from its ``*_workspace_bytes``; without one the
call allocates it.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Sequence, Union

import numpy as np
import torch

from . import _binding as zs
from . import tensors as zt

TRANSPOSE_A, TRANSPOSE_B = 1, 2     # ZS_TRANSPOSE_A, ZS_TRANSPOSE_B
NS_MAX_STEPS = 32                   # ZS_NS_MAX_STEPS
MATRIX_MAX_SIDE = 1 << 20           # ZS_MATRIX_MAX_SIDE
COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # the usual quintic

# every symbol include/zshard_matrices.h declares
MATRIX_EXPORTS = (
    "product_add_matrices_workspace_bytes", "product_add_matrices", "gram_add_matrices_workspace_bytes",
    "gram_add_matrices", "orthogonalize_matrices_workspace_bytes", "orthogonalize_matrices",
    "muon_step_matrices_workspace_bytes", "muon_step_matrices", "muon_scalars", "muon_step_matrices_dev",
)

_P, _I32, _I64, _D, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_float


class Product(ctypes.Structure):
    """zs_product"""
    _fields_ = [("a", _P), ("b", _P), ("c", _P), ("d", _P), ("m", _I64), ("n", _I64), ("k", _I64)]


class Gram(ctypes.Structure):
    """zs_gram"""
    _fields_ = [("a", _P), ("c", _P), ("d", _P), ("rows", _I64), ("cols", _I64), ("transposed", _I32),
                ("reserved", _I32)]


class Orthogonal(ctypes.Structure):
    """zs_orthogonal"""
    _fields_ = [("in", _P), ("out", _P), ("rows", _I64), ("cols", _I64)]


class Muon(ctypes.Structure):
    """zs_muon"""
    _fields_ = [(f, _D) for f in ("lr", "momentum", "weight_decay", "a", "b", "c", "eps", "grad_scale", "max_norm",
                                  "extra_norm_sq")] + [("nesterov", _I32), ("ns_steps", _I32)]


class MuonMatrix(ctypes.Structure):
    """zs_muon_matrix"""
    _fields_ = [("param", _P), ("grad", _P), ("momentum", _P), ("param_bf16", _P), ("rows", _I64), ("cols", _I64),
                ("scale", _D)]


class MuonScalars(ctypes.Structure):
    """zs_muon_scalars: one step's scalars as the kernels take them (64 bytes)."""
    _fields_ = [(f, _F) for f in ("momentum", "one_minus_momentum", "decay", "lr", "a", "b", "c", "grad_scale")] + \
               [("nesterov", _I32), ("clip", _I32), ("eps", _D), ("max_norm", _D), ("extra_norm_sq", _D)]


@dataclass
class MuonConfig:
    """Hyperparameters of one orthogonalised momentum step."""
    lr: float
    momentum: float = 0.95
    nesterov: bool = True
    weight_decay: float = 0.0
    ns_steps: int = 5
    coefficients: Sequence[float] = COEFFICIENTS
    eps: float = 1e-7
    grad_scale: float = 1.0
    max_norm: float = 0.0
    extra_norm_sq: float = 0.0

    def c_struct(self) -> Muon:
        a, b, c = self.coefficients
        return Muon(self.lr, self.momentum, self.weight_decay, a, b, c, self.eps, self.grad_scale, self.max_norm,
                    self.extra_norm_sq, int(bool(self.nesterov)), int(self.ns_steps))


_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    L = zs.lib()
    if _ready is not L:
        P, I32, I64, D = _P, _I32, _I64, _D
        for name, args, res in (
                ("product_add_matrices_workspace_bytes", [P, I32, I32, I32], I64),
                ("product_add_matrices", [P, I32, I32, I32, I32, I32, D, D, P, I64, P], I32),
                ("gram_add_matrices_workspace_bytes", [P, I32, I32], I64),
                ("gram_add_matrices", [P, I32, I32, I32, D, D, P, I64, P], I32),
                ("orthogonalize_matrices_workspace_bytes", [P, I32], I64),
                ("orthogonalize_matrices", [P, I32, I32, I32, D, D, D, D, P, I64, P], I32),
                ("muon_step_matrices_workspace_bytes", [P, I32], I64),
                ("muon_step_matrices", [ctypes.POINTER(Muon), P, I32, I32, I32, P, P, I64, P], I32),
                ("muon_scalars", [ctypes.POINTER(Muon), ctypes.POINTER(MuonScalars)], I32),
                ("muon_step_matrices_dev", [P, I32, P, I32, I32, I32, P, P, I64, P], I32)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _ready = L
    return L


# ---------------------------------------------------------------------------
# lists
# ---------------------------------------------------------------------------

def _matrices(ts, name: str) -> list:
    """The matrices of a list of 2-D and 3-D tensors."""
    out = []
    for k, t in enumerate(ts):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{k}]: expected a torch.Tensor")
        if t.dim() not in (2, 3):
            raise ValueError(f"{name}[{k}]: a matrix, or a stack of them, expected; got {t.dim()} dimensions")
        out += [t] if t.dim() == 2 else list(t.unbind(0))
    return out


def _stacks_as(ts, like, name: str) -> list:
    """_matrices, with None for every matrix of a tensor that is None."""
    if len(ts) != len(like):
        raise ValueError(f"{name}: {len(ts)} tensors, the list has {len(like)}")
    out = []
    for k, (t, p) in enumerate(zip(ts, like)):
        out += [None] * (1 if p.dim() == 2 else p.shape[0]) if t is None else _matrices([t], f"{name}[{k}]")
    return out


_FLOATS = (torch.float32, torch.bfloat16)


def _dtype(kind) -> int:
    return zs.ZS_BF16 if kind == torch.bfloat16 else zs.ZS_F32


class _MatrixList(zt._List):
    """A marshalled list of matrices of the given shapes."""

    def __init__(self, struct, shapes, device):
        self.count = len(shapes)
        self.shapes = [tuple(s) for s in shapes]
        self.numels = [r * c for r, c in self.shapes]
        self.array = np.zeros(max(self.count, 1), dtype=np.dtype(struct))
        self.address = self.array.ctypes.data
        self.device = device
        self.tensors = {}
        if any(max(s) > MATRIX_MAX_SIDE for s in self.shapes):
            raise ValueError(f"a matrix's sides are at most {MATRIX_MAX_SIDE}")

    def _put(self, field: str, name: str, ts, shapes, dtypes, optional: bool = False):
        """Device pointers of one kind of matrix, after the checks; its dtype."""
        if len(ts) != len(shapes):
            raise ValueError(f"{name}: {len(ts)} matrices, the list has {len(shapes)}")
        for k, (t, s) in enumerate(zip(ts, shapes)):
            if t is not None and tuple(t.shape) != tuple(s):
                raise ValueError(f"{name}[{k}]: {tuple(t.shape)} expected to be {tuple(s)}")
        pointers, kind = zt._pointers(ts, name, [r * c for r, c in shapes], dtypes, optional)
        self._set(field, ts, pointers)
        return kind

    def _fill(self, field: str, values) -> None:
        self.array[field][:self.count] = values


def _device(ts):
    return ts[0].device if ts else None


class ProductMatrices(_MatrixList):
    """The matrices of product_add_matrices: d = op(a) op(b) + c.  a, b: fp32 or
    bf16, one dtype; c (a list, or None) and d each of one dtype of either kind.
    c[k] may be d[k] itself."""

    def __init__(self, a, b, d, c=None, transpose_a: bool = False, transpose_b: bool = False):
        a, b, d = _matrices(a, "a"), _matrices(b, "b"), _matrices(d, "d")
        shapes = [tuple(t.shape) for t in d]
        super().__init__(Product, shapes, _device(d))
        if len(a) != self.count or len(b) != self.count:
            raise ValueError(f"{len(a)} a and {len(b)} b for {self.count} d")
        inner = [t.shape[0] if transpose_a else t.shape[1] for t in a]
        kind = self._put("a", "a", a, [(k, m) if transpose_a else (m, k) for (m, _), k in zip(shapes, inner)], _FLOATS)
        if self._put("b", "b", b, [(n, k) if transpose_b else (k, n) for (_, n), k in zip(shapes, inner)],
                     _FLOATS) != kind:
            raise TypeError("a and b must share one dtype")
        self.in_dtype = _dtype(kind)
        self.d_dtype = self.c_dtype = _dtype(self._put("d", "d", d, shapes, _FLOATS))
        if c is not None:
            self.c_dtype = _dtype(self._put("c", "c", _matrices(c, "c"), shapes, _FLOATS))
        self.flags = (TRANSPOSE_A if transpose_a else 0) | (TRANSPOSE_B if transpose_b else 0)
        for field, values in (("m", [m for m, _ in shapes]), ("n", [n for _, n in shapes]), ("k", inner)):
            self._fill(field, values)


class GramMatrices(_MatrixList):
    """The matrices of gram_add_matrices: d = a a^T + c, or a^T a + c where d has
    a's columns as its side.  transposed: for a square a both fit, and a a^T is
    taken unless it is True (one value, or one per tensor of a; None: by d's side).
    a: fp32 or bf16; c (a list, or None) and d: one dtype.  c[k] may be d[k] itself."""

    def __init__(self, a, d, c=None, transposed: Union[None, bool, Sequence[Optional[bool]]] = None):
        a = list(a)
        asked = [transposed] * len(a) if transposed is None or np.isscalar(transposed) else list(transposed)
        if len(asked) != len(a):
            raise ValueError(f"transposed: {len(asked)} values for {len(a)} tensors")
        asked = [x for t, x in zip(a, asked)
                 for _ in range(t.shape[0] if isinstance(t, torch.Tensor) and t.dim() == 3 else 1)]
        a, d = _matrices(a, "a"), _matrices(d, "d")
        super().__init__(Gram, [tuple(t.shape) for t in d], _device(d))
        self.in_dtype = _dtype(self._put("a", "a", a, [tuple(t.shape) for t in a], _FLOATS))
        if len(a) != self.count:
            raise ValueError(f"{len(a)} a for {self.count} d")
        turned = []
        for k, (t, s, x) in enumerate(zip(a, self.shapes, asked)):
            if s not in ((t.shape[0],) * 2, (t.shape[1],) * 2):
                raise ValueError(f"d[{k}]: {s} is neither side of a[{k}], {tuple(t.shape)}")
            turned.append(int(s[0] != t.shape[0]) if x is None else int(bool(x)))
            if s[0] != t.shape[turned[-1]]:
                raise ValueError(f"d[{k}]: {s}, but a[{k}] is {tuple(t.shape)} and transposed {bool(x)}")
        kind = self._put("d", "d", d, self.shapes, _FLOATS)
        self.d_dtype = _dtype(kind)
        if c is not None and self.count and self._put("c", "c", _matrices(c, "c"), self.shapes, _FLOATS) != kind:
            raise TypeError("c and d must share one dtype")
        for field, values in (("rows", [t.shape[0] for t in a]), ("cols", [t.shape[1] for t in a]),
                              ("transposed", turned)):
            self._fill(field, values)


class OrthogonalizeMatrices(_MatrixList):
    """The matrices of orthogonalize_matrices: inputs (fp32 or bf16, one dtype)
    and outputs (bf16) of the same shapes."""

    def __init__(self, inputs, outputs):
        inputs, outputs = _matrices(inputs, "inputs"), _matrices(outputs, "outputs")
        super().__init__(Orthogonal, [tuple(t.shape) for t in inputs], _device(inputs))
        self.in_dtype = _dtype(self._put("in", "inputs", inputs, self.shapes, _FLOATS))
        self._put("out", "outputs", outputs, self.shapes, (torch.bfloat16,))
        for field, i in (("rows", 0), ("cols", 1)):
            self._fill(field, [s[i] for s in self.shapes])


def update_scale(rows: int, cols: int, scale: Union[str, float] = "rms") -> float:
    """A matrix's factor of the learning rate: "rms" 0.2 sqrt(max(rows, cols)),
    which gives an update the RMS that AdamW's usually has; "spectral"
    sqrt(max(1, rows / cols)); or a number."""
    if scale == "rms":
        return 0.2 * math.sqrt(max(rows, cols))
    if scale == "spectral":
        return math.sqrt(max(1.0, rows / cols)) if cols else 1.0
    if isinstance(scale, str):
        raise ValueError(f"scale: 'rms', 'spectral' or a number, got {scale!r}")
    return float(scale)


class MuonMatrices(_MatrixList):
    """The matrices of muon_step_matrices: params (fp32 or bf16), grads (fp32 or
    bf16), momenta (fp32), and for fp32 params their bf16 re-casts (a list with
    None where a tensor has none, or None).  scale: as update_scale takes it, or
    one per tensor."""

    def __init__(self, params, grads, momenta, param_bf16=None, scale="rms"):
        params = list(params)
        scales = [scale] * len(params) if isinstance(scale, str) or np.isscalar(scale) else list(scale)
        if len(scales) != len(params):
            raise ValueError(f"scale: {len(scales)} values for {len(params)} tensors")
        matrices = _matrices(params, "params")
        super().__init__(MuonMatrix, [tuple(t.shape) for t in matrices], _device(matrices))
        self.param_dtype = _dtype(self._put("param", "params", matrices, self.shapes, _FLOATS))
        self.set_grads(grads)
        self._put("momentum", "momenta", _matrices(momenta, "momenta"), self.shapes, (torch.float32,))
        if param_bf16 is not None and any(t is not None for t in param_bf16):
            if self.param_dtype == zs.ZS_BF16:
                raise ValueError("param_bf16: a re-cast of fp32 parameters; these are bf16")
            self._put("param_bf16", "param_bf16", _stacks_as(list(param_bf16), params, "param_bf16"), self.shapes,
                      (torch.bfloat16,), optional=True)
        for field, i in (("rows", 0), ("cols", 1)):
            self._fill(field, [s[i] for s in self.shapes])
        factors = [update_scale(*(p.shape[-2:]), s) for p, s in zip(params, scales)
                   for _ in range(1 if p.dim() == 2 else p.shape[0])]
        if not all(math.isfinite(_F(s).value) for s in factors):
            raise ValueError("scale: finite values, in binary32 too")
        self._fill("scale", factors)

    def set_grads(self, grads) -> None:
        """Other gradients of the same shapes (fp32 or bf16, one dtype)."""
        self.grad_dtype = _dtype(self._put("grad", "grads", _matrices(grads, "grads"), self.shapes, _FLOATS))


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def _need(fn: str, n: int) -> int:
    if n < 0:
        raise ValueError(f"{fn}: invalid list")
    return n


def _workspace(workspace: Optional[torch.Tensor], need: int, lst: _MatrixList, stream):
    """Address, bytes and the tensor itself; allocated on the stream where none is given."""
    if workspace is None:
        # of the stream it is used on: freed at return, it is next used in that stream's order
        with torch.cuda.stream(stream):
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=lst.device)
    return zs._dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), workspace


def product_add_matrices_workspace_bytes(products: ProductMatrices) -> int:
    fn = "product_add_matrices_workspace_bytes"
    return _need(fn, int(_lib().product_add_matrices_workspace_bytes(products.address, products.count,
                                                                     products.in_dtype, products.flags)))


def product_add_matrices(products: ProductMatrices, alpha: float = 1.0, beta: float = 1.0,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """d = alpha * op(a) op(b) + beta * c for every entry of the list."""
    products.check("product_add_matrices")
    if not products.count:
        return
    at, size, held = _workspace(workspace, product_add_matrices_workspace_bytes(products), products, stream)
    zs._check("product_add_matrices", _lib().product_add_matrices(
        products.address, products.count, products.in_dtype, products.c_dtype, products.d_dtype, products.flags,
        float(alpha), float(beta), at, size, zs._stream(stream)))


def gram_add_matrices_workspace_bytes(grams: GramMatrices) -> int:
    fn = "gram_add_matrices_workspace_bytes"
    return _need(fn, int(_lib().gram_add_matrices_workspace_bytes(grams.address, grams.count, grams.in_dtype)))


def gram_add_matrices(grams: GramMatrices, alpha: float = 1.0, beta: float = 1.0,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """d = alpha * a a^T (or a^T a) + beta * c for every entry of the list; c symmetric."""
    grams.check("gram_add_matrices")
    if not grams.count:
        return
    at, size, held = _workspace(workspace, gram_add_matrices_workspace_bytes(grams), grams, stream)
    zs._check("gram_add_matrices", _lib().gram_add_matrices(
        grams.address, grams.count, grams.in_dtype, grams.d_dtype, float(alpha), float(beta), at, size,
        zs._stream(stream)))


def orthogonalize_matrices_workspace_bytes(matrices: OrthogonalizeMatrices) -> int:
    fn = "orthogonalize_matrices_workspace_bytes"
    return _need(fn, int(_lib().orthogonalize_matrices_workspace_bytes(matrices.address, matrices.count)))


def orthogonalize_matrices(matrices: OrthogonalizeMatrices, steps: int = 5, coefficients=COEFFICIENTS,
                           eps: float = 1e-7, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Every output: its input, divided by its Frobenius norm and put through
    `steps` Newton-Schulz steps X <- a X + (b S + c S^2) X, S = X X^T."""
    matrices.check("orthogonalize_matrices")
    if not matrices.count:
        return
    a, b, c = coefficients
    at, size, held = _workspace(workspace, orthogonalize_matrices_workspace_bytes(matrices), matrices, stream)
    zs._check("orthogonalize_matrices", _lib().orthogonalize_matrices(
        matrices.address, matrices.count, matrices.in_dtype, int(steps), float(a), float(b), float(c), float(eps), at,
        size, zs._stream(stream)))


def muon_step_matrices_workspace_bytes(matrices: MuonMatrices) -> int:
    fn = "muon_step_matrices_workspace_bytes"
    return _need(fn, int(_lib().muon_step_matrices_workspace_bytes(matrices.address, matrices.count)))


def muon_step_matrices(hp: MuonConfig, matrices: MuonMatrices, norm_sq: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The orthogonalised momentum update of every matrix of the list (in place)."""
    matrices.check("muon_step_matrices")
    c = hp.c_struct()
    if not matrices.count:
        return
    at, size, held = _workspace(workspace, muon_step_matrices_workspace_bytes(matrices), matrices, stream)
    zs._check("muon_step_matrices", _lib().muon_step_matrices(
        ctypes.byref(c), matrices.address, matrices.count, matrices.param_dtype, matrices.grad_dtype,
        zs._norm(norm_sq, "muon_step_matrices"), at, size, zs._stream(stream)))


def muon_scalars_bytes(hp: MuonConfig) -> bytes:
    """muon_scalars(hp) as the bytes muon_step_matrices_dev reads."""
    out, c = MuonScalars(), hp.c_struct()
    zs._check("muon_scalars", _lib().muon_scalars(ctypes.byref(c), ctypes.byref(out)))
    return bytes(out)


def muon_step_matrices_dev(scalars_dev: torch.Tensor, ns_steps: int, matrices: MuonMatrices,
                           norm_sq: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """muon_step_matrices with its scalars read from device memory when the
    kernels run (scalars_dev: uint8 GPU tensor holding muon_scalars_bytes(hp))."""
    matrices.check("muon_step_matrices_dev")
    if not matrices.count:
        return
    at, size, held = _workspace(workspace, muon_step_matrices_workspace_bytes(matrices), matrices, stream)
    zs._check("muon_step_matrices_dev", _lib().muon_step_matrices_dev(
        zt._scalars_dev(scalars_dev, MuonScalars, "muon_step_matrices_dev"), int(ns_steps), matrices.address,
        matrices.count, matrices.param_dtype, matrices.grad_dtype, zs._norm(norm_sq, "muon_step_matrices_dev"), at, size,
        zs._stream(stream)))
