"""The calls over lists of matrices and of mixed precision on the host: exports,
sizes and refusals.

No call reaches a launch (there is no GPU here): each fails validation or has
nothing to do.  Pointers passed are never dereferenced.
"""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import fsdp_sharded_optimizer_amd as zs
from fsdp_sharded_optimizer_amd import _binding as B
from fsdp_sharded_optimizer_amd import matrices as M
from fsdp_sharded_optimizer_amd import tensors as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
MIB = 1 << 20
GIB = 1 << 30
L = M._lib()
T._lib()


@pytest.fixture(autouse=True)
def no_launch_reached():
    yield
    assert zs.lib().zs_last_hip_error() == 0, "a call got past validation to a kernel launch"


def fill(struct, rows):
    a = (struct * max(len(rows), 1))()
    for k, row in enumerate(rows):
        for name, value in zip((f for f, _ in struct._fields_), row):
            setattr(a[k], name, value)
    return a


def edited(rows, k, j, value):
    rows = [list(r) for r in rows]
    rows[k][j] = value
    return rows


def test_exports_match_the_header():
    text = open(os.path.join(ROOT, "include", "zshard_matrices.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*ZS_API\s+(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", text, flags=re.M))
    assert names == set(zs.MATRIX_EXPORTS)
    for name in names:
        assert getattr(L, name) is not None


def test_header_is_plain_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src = tmp_path / "c.c"
    src.write_text('#include "zshard_matrices.h"\n#include "zshard_tensors.h"\n#include <stdio.h>\nint main(void) {\n'
                   "  zs_muon hp = {.lr = 1e-3, .momentum = 0.95, .a = 3.4445, .b = -4.775, .c = 2.0315, .eps = 1e-7,"
                   " .grad_scale = 1.0, .nesterov = 1, .ns_steps = 5};\n"
                   "  zs_muon_scalars sc; zs_muon_matrix m = {0}; zs_mixed_tensor t = {0};\n"
                   "  m.rows = 100; m.cols = 300; t.numel = 5; t.dtype = ZS_BF16;\n"
                   "  if (muon_scalars(&hp, &sc) != ZS_OK || sizeof sc != 64) return 1;\n"
                   "  if (muon_step_matrices(&hp, NULL, 0, ZS_F32, ZS_BF16, NULL, NULL, 0, NULL) != ZS_OK) return 2;\n"
                   "  if (grad_clip_tensors(NULL, NULL, 0, 1.0, 1.0, 0.0, NULL, NULL) != ZS_OK) return 3;\n"
                   '  printf("%lld %lld\\n", (long long)muon_step_matrices_workspace_bytes(&m, 1),\n'
                   "         (long long)grad_norms_sq_tensors_workspace_bytes(&t, 1));\n  return 0;\n}\n")
    exe = str(tmp_path / "c")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Wextra", "-Wpedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-o", exe, str(src), B.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(B.LIB_PATH)}"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    need = L.muon_step_matrices_workspace_bytes(fill(M.MuonMatrix, [[0, 0, 0, 0, 100, 300, 1.0]]), 1)
    assert out.returncode == 0 and out.stdout.split() == [str(need), "16"]


# --- lists of mixed precision ---------------------------------------------------

def test_mixed_norms_reject():
    good = [[FAKE, 5000, 0, 0], [FAKE + MIB, 300, 1, 0]]
    out, norms, ws = FAKE + 2 * MIB, FAKE + 3 * MIB, FAKE + 4 * MIB

    def f(rows, count=None, scale=1.0, o=out, e=norms, w=ws, nbytes=MIB):
        return L.grad_norms_sq_tensors(fill(T.MixedTensor, rows), len(rows) if count is None else count, scale, e, o, w,
                                       nbytes, None)

    def need(rows):
        return L.grad_norms_sq_tensors_workspace_bytes(fill(T.MixedTensor, rows), len(rows))
    assert need([]) == 0 and need([[0, 0, 0, 0]]) == 8
    assert need([[0, 4097, 0, 0], [0, 8193, 1, 0]]) == (2 + 2 + 2) * 8
    for j, value in ((1, -1), (1, (1 << 35) + 1), (2, 2), (2, -1), (3, 1)):
        assert f(edited(good, 1, j, value)) == B.ZS_EINVAL and need(edited(good, 1, j, value)) == -1
    assert f(good, count=-1) == B.ZS_EINVAL
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert f(good, scale=scale) == B.ZS_EINVAL
    assert f(good, o=None) == B.ZS_EINVAL and f(good, o=out + 4) == B.ZS_EINVAL and f(good, e=norms + 4) == B.ZS_EINVAL
    assert f(good, w=None) == B.ZS_EINVAL and f(good, w=ws + 4) == B.ZS_EINVAL
    assert f(good, nbytes=need(good) - 1) == B.ZS_EWORKSPACE
    assert f(edited(good, 1, 0, 0)) == B.ZS_EINVAL and f(edited(good, 0, 0, FAKE + 2)) == B.ZS_EINVAL
    assert f(edited(good, 1, 0, FAKE + MIB + 1)) == B.ZS_EINVAL
    assert f(good, o=FAKE + 80) == B.ZS_EOVERLAP and f(good, w=FAKE + 80) == B.ZS_EOVERLAP
    assert f(good, e=FAKE + 80) == B.ZS_EOVERLAP and f(good, e=out) == B.ZS_EOVERLAP
    assert f(good, w=out) == B.ZS_EOVERLAP and f(good, w=norms) == B.ZS_EOVERLAP
    assert L.grad_norms_sq_tensors(None, 1, 1.0, None, out, ws, MIB, None) == B.ZS_EINVAL


def test_clip_rejects():
    good = [[FAKE, 5000, 0, 0], [FAKE + MIB, 300, 1, 0]]
    to = [[FAKE + 2 * MIB, 5000, 1, 0], [FAKE + 3 * MIB, 300, 0, 0]]
    norm = FAKE + 4 * MIB

    def f(a, b, count=None, scale=1.0, most=1.0, extra=0.0, n=norm):
        return L.grad_clip_tensors(fill(T.MixedTensor, a), fill(T.MixedTensor, b), len(a) if count is None else count,
                                   scale, most, extra, n, None)
    assert f([], []) == B.ZS_OK and f([[0, 0, 0, 0]], [[0, 0, 1, 0]]) == B.ZS_OK
    assert f(good, to, count=-1) == B.ZS_EINVAL
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(most=float("nan")), dict(extra=-1.0),
               dict(extra=float("nan")), dict(n=norm + 4)):
        assert f(good, to, **kw) == B.ZS_EINVAL, kw
    for rows, other in ((good, to), (to, good)):
        for j, value in ((0, 0), (1, 301), (2, 2), (3, 7)):
            bad = edited(rows, 1, j, value)
            assert (f(bad, other) if rows is good else f(other, bad)) == B.ZS_EINVAL, (j, value)
    assert f(edited(good, 0, 0, FAKE + 2), to) == B.ZS_EINVAL and f(good, edited(to, 0, 0, FAKE + 2 * MIB + 1)) == B.ZS_EINVAL
    # in place: the same dtype and the very same memory
    assert f(good, edited(to, 0, 0, FAKE)) == B.ZS_EOVERLAP              # bf16 over fp32
    assert f(good, edited(edited(to, 0, 2, 0), 0, 0, FAKE + 4)) == B.ZS_EOVERLAP
    assert f(good, edited(to, 1, 0, FAKE + 2 * MIB)) == B.ZS_EOVERLAP    # two results in one place
    assert f([good[0], good[0]], [good[0], [FAKE + MIB, 5000, 0, 0]]) == B.ZS_EOVERLAP   # read and written
    assert f(good, to, n=FAKE + 2 * MIB + 8) == B.ZS_EOVERLAP


# --- products ---------------------------------------------------------------------

def products(m=100, n=90, k=70, count=2):
    """Disjoint buffers, 1 MiB apart: (a, b, c, d, m, n, k)."""
    return [[FAKE + (4 * i + j) * MIB for j in range(4)] + [m, n, k] for i in range(count)]


WS = FAKE + 64 * MIB


def product(rows, count=None, i=1, c=0, d=0, flags=0, alpha=1.0, beta=1.0, ws=WS, nbytes=GIB):
    return L.product_add_matrices(fill(M.Product, rows), len(rows) if count is None else count, i, c, d, flags, alpha,
                                  beta, ws, nbytes, None)


def product_need(rows, i=1, flags=0):
    return L.product_add_matrices_workspace_bytes(fill(M.Product, rows), len(rows), i, flags)


BAD_SHAPES = [(4, -1), (4, (1 << 20) + 1), (5, -1), (6, -1), (6, (1 << 20) + 1)]


def test_products_reject():
    good = products()
    assert product([]) == B.ZS_OK and product(products(0)) == B.ZS_OK and product(products(5, 0)) == B.ZS_OK
    assert product([[0, 0, 0, 0, 0, 7, 9]]) == B.ZS_OK                    # without elements: pointers are not looked at
    for j, value in BAD_SHAPES:
        assert product(edited(good, 1, j, value)) == B.ZS_EINVAL and product_need(edited(good, 1, j, value)) == -1
    for sides in ((1 << 16, 1 << 16, 1), (1 << 16, 1, 1 << 16), (1, 1 << 16, 1 << 16)):
        assert product([good[0][:4] + list(sides)]) == B.ZS_EINVAL        # 2^32 elements
    assert product(good, count=-1) == B.ZS_EINVAL
    assert L.product_add_matrices(None, 1, 1, 0, 0, 0, 1.0, 1.0, WS, GIB, None) == B.ZS_EINVAL
    for kw in (dict(i=2), dict(c=2), dict(d=-1), dict(flags=4), dict(alpha=float("nan")), dict(beta=float("inf"))):
        assert product(good, **kw) == B.ZS_EINVAL, kw
    for j in (0, 1, 3):
        assert product(edited(good, 1, j, 0)) == B.ZS_EINVAL, j
    for j, kw in ((0, dict(i=0)), (1, dict(i=0)), (2, {}), (3, {})):
        assert product(edited(good, 1, j, good[1][j] + 2), **kw) == B.ZS_EINVAL, j
    assert product(good, ws=None) == B.ZS_EINVAL and product(good, ws=WS + 128) == B.ZS_EINVAL
    assert product(good, nbytes=product_need(good) - 1) == B.ZS_EWORKSPACE
    for j in (0, 1):
        assert product(edited(good, 1, 3, good[0][j] + 16)) == B.ZS_EOVERLAP
        assert product(good, ws=good[1][j]) == B.ZS_EOVERLAP
    assert product(edited(good, 1, 3, good[0][3])) == B.ZS_EOVERLAP       # one result twice
    assert product(edited(good, 0, 2, good[0][3] + 4)) == B.ZS_EOVERLAP   # c beside d
    assert product(edited(good, 0, 2, good[0][3]), c=1) == B.ZS_EOVERLAP  # c is d, of another dtype
    assert product(edited(good, 1, 2, good[0][3])) == B.ZS_EOVERLAP       # another entry's result
    assert product(good, ws=good[1][3]) == B.ZS_EOVERLAP


def test_products_workspace():
    lies = products(100, 88, 128)
    assert product_need(lies) == 0 and product_need(lies, flags=2) == 0
    pad = lambda r, c: 2 * (-(-r // 64) * 64) * (-(-c // 64) * 64)  # noqa: E731
    assert product_need(lies, flags=1) == 2 * pad(100, 128)                # a transposed
    assert product_need(products(100, 90, 128)) == 2 * pad(90, 128)        # b's rows are not whole chunks
    assert product_need(products(100, 90, 128), flags=2) == 0
    assert product_need(products(100, 88, 70)) == 2 * (pad(100, 70) + pad(88, 70))
    assert product_need(edited(lies, 0, 0, FAKE + 2)) == pad(100, 128)     # off a 16-byte boundary
    assert product_need(lies, i=0) == 6 * (pad(100, 128) + pad(88, 128))
    assert product_need(products(100, 90, 0)) == 0


def grams(rows=100, cols=70, turned=0, count=2):
    return [[FAKE + (3 * i + j) * MIB for j in range(3)] + [rows, cols, turned, 0] for i in range(count)]


def gram(rows, count=None, i=1, d=0, alpha=1.0, beta=1.0, ws=WS, nbytes=GIB):
    return L.gram_add_matrices(fill(M.Gram, rows), len(rows) if count is None else count, i, d, alpha, beta, ws, nbytes,
                               None)


def test_grams_reject():
    good = grams()
    need = L.gram_add_matrices_workspace_bytes(fill(M.Gram, good), 2, 1)
    assert need == 2 * 2 * 128 * 128
    assert L.gram_add_matrices_workspace_bytes(fill(M.Gram, grams(100, 128)), 2, 1) == 0
    assert L.gram_add_matrices_workspace_bytes(fill(M.Gram, grams(100, 128, 1)), 2, 1) == 2 * 2 * 128 * 128
    assert L.gram_add_matrices_workspace_bytes(fill(M.Gram, grams(100, 128)), 2, 0) == 2 * 2 * 3 * 2 * 128 * 128
    assert gram([]) == B.ZS_OK and gram(grams(0, 5)) == B.ZS_OK
    for j, value in ((3, -1), (4, (1 << 20) + 1), (5, 2), (5, -1), (6, 1)):
        assert gram(edited(good, 1, j, value)) == B.ZS_EINVAL
    assert gram([good[0][:3] + [1 << 16, 4, 0, 0]]) == B.ZS_EINVAL         # a result of 2^32 elements
    assert gram(good, count=-1) == B.ZS_EINVAL
    for kw in (dict(i=2), dict(d=3), dict(alpha=float("inf")), dict(beta=float("nan"))):
        assert gram(good, **kw) == B.ZS_EINVAL, kw
    assert gram(edited(good, 1, 0, 0)) == B.ZS_EINVAL and gram(edited(good, 1, 2, 0)) == B.ZS_EINVAL
    assert gram(edited(good, 1, 1, good[1][1] + 2)) == B.ZS_EINVAL
    assert gram(good, nbytes=need - 1) == B.ZS_EWORKSPACE and gram(good, ws=None) == B.ZS_EINVAL
    assert gram(edited(good, 1, 2, good[0][0])) == B.ZS_EOVERLAP and gram(edited(good, 1, 2, good[0][2])) == B.ZS_EOVERLAP
    assert gram(edited(good, 1, 1, good[0][2])) == B.ZS_EOVERLAP and gram(good, ws=good[0][2]) == B.ZS_EOVERLAP


# --- orthogonalisation and the step ---------------------------------------------------

def orthogonals(rows=100, cols=70, count=2):
    return [[FAKE + (2 * i + j) * MIB for j in range(2)] + [rows, cols] for i in range(count)]


def orthogonalize(rows, count=None, i=1, steps=5, abc=(3.4445, -4.775, 2.0315), eps=1e-7, ws=WS, nbytes=GIB):
    return L.orthogonalize_matrices(fill(M.Orthogonal, rows), len(rows) if count is None else count, i, steps, *abc, eps,
                                    ws, nbytes, None)


def test_orthogonalize_rejects():
    good = orthogonals()
    need = L.orthogonalize_matrices_workspace_bytes(fill(M.Orthogonal, good), 2)
    assert orthogonalize([]) == B.ZS_OK and orthogonalize(orthogonals(0)) == B.ZS_OK
    for j, value in ((2, -1), (3, (1 << 20) + 1)):
        assert orthogonalize(edited(good, 1, j, value)) == B.ZS_EINVAL
    assert orthogonalize([good[0][:2] + [1 << 16, 1 << 16]]) == B.ZS_EINVAL
    assert orthogonalize(good, count=-1) == B.ZS_EINVAL
    for kw in (dict(i=2), dict(steps=0), dict(steps=33), dict(abc=(33.0, 0.0, 0.0)), dict(abc=(1.0, float("nan"), 0.0)),
               dict(abc=(1.0, 0.0, float("-inf"))), dict(eps=0.0), dict(eps=1e-31), dict(eps=float("inf")), dict(eps=float("nan"))):
        assert orthogonalize(good, **kw) == B.ZS_EINVAL, kw
    for j in (0, 1):
        assert orthogonalize(edited(good, 1, j, 0)) == B.ZS_EINVAL
        assert orthogonalize(edited(good, 1, j, good[1][j] + 1)) == B.ZS_EINVAL
    assert orthogonalize(edited(good, 1, 0, good[1][0] + 2), i=0) == B.ZS_EINVAL
    assert orthogonalize(good, nbytes=need - 1) == B.ZS_EWORKSPACE
    assert orthogonalize(good, ws=None) == B.ZS_EINVAL and orthogonalize(good, ws=WS + 64) == B.ZS_EINVAL
    assert orthogonalize(edited(good, 1, 1, good[1][0])) == B.ZS_EOVERLAP    # in place
    assert orthogonalize(edited(good, 1, 1, good[0][1] + 2)) == B.ZS_EOVERLAP
    assert orthogonalize(good, ws=good[0][0]) == B.ZS_EOVERLAP and orthogonalize(good, ws=good[1][1]) == B.ZS_EOVERLAP


def test_workspace_is_shared_by_groups():
    def need(*shapes):
        return L.orthogonalize_matrices_workspace_bytes(fill(M.Orthogonal, [[0, 0, r, c] for r, c in shapes]), len(shapes))
    assert need() == 0 and need((0, 5)) == 0
    one = need((4096, 11008))
    # X's two halves twice, S and a polynomial of it: 4 + 2 * 4096 / 11008 = 4.744 times the matrix in 16 bits
    assert 4.74 * 2 * 4096 * 11008 < one < 4.75 * 2 * 4096 * 11008
    assert need(*[(4096, 11008)] * 100) < 11.1 * one     # 2^29 elements: 11 of them
    assert need((100, 300), (300, 100)) < 2 * need((100, 300)) and need((100, 300)) == need((300, 100))
    for bad in ((-1, 5), (1 << 21, 1), (1 << 16, 1 << 16)):
        assert need((100, 100), bad) == -1


HP = dict(lr=1e-3, momentum=0.95, weight_decay=0.1, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, grad_scale=1.0, max_norm=1.0,
          extra_norm_sq=0.0, nesterov=1, ns_steps=5)
BAD_HP = [dict(lr=-1.0), dict(lr=float("inf")), dict(lr=float("nan")), dict(momentum=1.0), dict(momentum=-0.1),
          dict(weight_decay=-1.0), dict(a=33.0), dict(b=float("nan")), dict(c=-33.0), dict(eps=0.0), dict(eps=float("nan")),
          dict(grad_scale=0.0), dict(max_norm=float("nan")), dict(extra_norm_sq=-1.0), dict(extra_norm_sq=float("nan")),
          dict(nesterov=2), dict(nesterov=-1), dict(ns_steps=0), dict(ns_steps=33)]


def hp_with(**kw):
    h = M.Muon()
    for name, value in {**HP, **kw}.items():
        setattr(h, name, value)
    return ctypes.byref(h)


def muons(rows=100, cols=70, count=2):
    return [[FAKE + (4 * i + j) * MIB for j in range(4)] + [rows, cols, 1.5] for i in range(count)]


def muon(rows, h=None, count=None, p=0, g=1, norm=None, ws=WS, nbytes=GIB):
    return L.muon_step_matrices(h if h is not None else hp_with(), fill(M.MuonMatrix, rows),
                                len(rows) if count is None else count, p, g, norm, ws, nbytes, None)


def muon_dev(rows, sc=FAKE - 64, steps=5, p=0, g=1, norm=None):
    return L.muon_step_matrices_dev(sc, steps, fill(M.MuonMatrix, rows), len(rows), p, g, norm, WS, GIB, None)


def test_muon_rejects():
    good = muons()
    need = L.muon_step_matrices_workspace_bytes(fill(M.MuonMatrix, good), 2)
    assert need == L.orthogonalize_matrices_workspace_bytes(fill(M.Orthogonal, orthogonals()), 2)
    assert muon([]) == B.ZS_OK and muon(muons(0)) == B.ZS_OK and muon([[0, 0, 0, 0, 0, 3, 1.0]]) == B.ZS_OK
    out = M.MuonScalars()
    for bad in BAD_HP:
        assert muon(good, h=hp_with(**bad)) == B.ZS_EINVAL, bad
        assert L.muon_scalars(hp_with(**bad), ctypes.byref(out)) == B.ZS_EINVAL, bad
    assert L.muon_step_matrices(None, fill(M.MuonMatrix, good), 2, 0, 1, None, WS, GIB, None) == B.ZS_EINVAL
    assert L.muon_scalars(hp_with(), None) == B.ZS_EINVAL and L.muon_scalars(None, ctypes.byref(out)) == B.ZS_EINVAL
    assert muon(good, count=-1) == B.ZS_EINVAL and muon(good, p=2) == B.ZS_EINVAL and muon(good, g=-1) == B.ZS_EINVAL
    for j in (0, 1, 2):
        assert muon(edited(good, 1, j, 0)) == B.ZS_EINVAL
    for j, step in ((0, 2), (1, 1), (2, 2), (3, 1)):
        assert muon(edited(good, 1, j, good[1][j] + step)) == B.ZS_EINVAL
    assert muon(good, p=1) == B.ZS_EINVAL                                   # a re-cast of bf16 parameters
    for j, value in ((4, -1), (5, (1 << 20) + 1), (6, float("inf")), (6, float("nan")), (6, 1e39)):
        assert muon(edited(good, 1, j, value)) == B.ZS_EINVAL
    assert muon(good, norm=FAKE - 4) == B.ZS_EINVAL
    assert muon_dev(good, sc=None) == B.ZS_EINVAL and muon_dev(good, sc=FAKE - 60) == B.ZS_EINVAL
    assert muon_dev(good, steps=0) == B.ZS_EINVAL and muon_dev(good, steps=33) == B.ZS_EINVAL
    assert muon(good, nbytes=need - 1) == B.ZS_EWORKSPACE and muon(good, ws=None) == B.ZS_EINVAL
    for a in range(4):
        for b in range(a):
            assert muon(edited(good, 0, a, good[0][b] + 16)) == B.ZS_EOVERLAP, (a, b)
            assert muon(edited(good, 1, a, good[0][b] + 16)) == B.ZS_EOVERLAP, (a, b)
        if a != 1:
            assert muon(good, norm=good[1][a] + 8) == B.ZS_EOVERLAP
            assert muon_dev(good, sc=good[1][a] + 8) == B.ZS_EOVERLAP
        assert muon(good, ws=good[1][a]) == B.ZS_EOVERLAP


def test_muon_scalars():
    raw = zs.muon_scalars_bytes(zs.MuonConfig(lr=0.01, momentum=0.9, weight_decay=0.5, grad_scale=0.25, max_norm=2.0,
                                              extra_norm_sq=3.0, nesterov=False))
    sc = M.MuonScalars.from_buffer_copy(raw)
    f = lambda x: ctypes.c_float(x).value  # noqa: E731
    assert len(raw) == 64
    assert (sc.momentum, sc.one_minus_momentum, sc.decay, sc.lr) == (f(0.9), f(1 - 0.9), f(1 - 0.005), f(0.01))
    assert (sc.a, sc.b, sc.c, sc.grad_scale) == (f(3.4445), f(-4.775), f(2.0315), 0.25)
    assert (sc.nesterov, sc.clip, sc.eps, sc.max_norm, sc.extra_norm_sq) == (0, 1, 1e-7, 2.0, 3.0)


def test_update_scale():
    assert zs.update_scale(100, 400) == zs.update_scale(400, 100) == 0.2 * 20
    assert zs.update_scale(400, 100, "spectral") == 2.0 and zs.update_scale(100, 400, "spectral") == 1.0
    assert zs.update_scale(3, 4, 0.5) == 0.5
    with pytest.raises(ValueError):
        zs.update_scale(3, 4, "no")


def test_lists_refuse_what_cannot_be_marshalled():
    x = torch.zeros(4, 4)
    makes = (lambda: zs.ProductMatrices([x], [x], [x]), lambda: zs.GramMatrices([x], [x]),
             lambda: zs.OrthogonalizeMatrices([x], [x]), lambda: zs.MuonMatrices([x], [x], [x]),
             lambda: zs.MixedTensors([x]), lambda: zs.MuonOptimizer([x], lr=0.1))
    for make in makes:
        with pytest.raises(ValueError, match="GPU tensor"):
            make()
    for bad in (torch.zeros(4), torch.zeros(2, 2, 2, 2)):
        with pytest.raises(ValueError, match="dimensions"):
            zs.OrthogonalizeMatrices([bad], [bad])
    with pytest.raises(TypeError):
        zs.GramMatrices([None], [x])
    with pytest.raises(ValueError):
        zs.OrthogonalizeMatrices([x], [x, x])
    with pytest.raises(ValueError):
        zs.OrthogonalizeMatrices([x], [torch.zeros(2, 8)])
    with pytest.raises(ValueError):
        zs.MuonMatrices([x], [x], [x], scale=[1.0, 2.0])


def test_scalars_beyond_the_kernels_range_are_refused():
    """Finite in binary64 and infinite in the binary32 that the kernels hold."""
    rows, grams = [[FAKE, FAKE + MIB, 0, FAKE + 2 * MIB, 64, 64, 64]], [[FAKE, 0, FAKE + MIB, 64, 64, 0, 0]]
    for kw in (dict(alpha=1e39), dict(alpha=-1e300), dict(beta=1e39)):
        assert product(rows, **kw) == B.ZS_EINVAL and gram(grams, **kw) == B.ZS_EINVAL, kw
    out = M.MuonScalars()
    for kw in (dict(lr=1e39), dict(grad_scale=1e39), dict(lr=1e20, weight_decay=1e20), dict(weight_decay=float("inf")),
               dict(weight_decay=float("nan"))):
        assert muon(muons(), h=hp_with(**kw)) == B.ZS_EINVAL, kw
        assert L.muon_scalars(hp_with(**kw), ctypes.byref(out)) == B.ZS_EINVAL, kw
    assert L.muon_scalars(hp_with(lr=1e38, weight_decay=1.0), ctypes.byref(out)) == B.ZS_OK


def test_grad_scales_that_binary32_does_not_hold_are_refused():
    """The kernels multiply by the binary32 value: an infinite one would write inf and NaN over
    the gradients, one that is 0 there would erase them."""
    grads = fill(T.MixedTensor, [[FAKE, 5000, 0, 0]])
    for scale in (1e39, 1e300, 1e-46, 1e-60, 5e-324):
        assert L.grad_clip_tensors(grads, grads, 1, scale, 0.0, 0.0, None, None) == B.ZS_EINVAL
        assert L.grad_norms_sq_tensors(grads, 1, scale, None, FAKE + MIB, FAKE + 2 * MIB, MIB, None) == B.ZS_EINVAL
        with pytest.raises(zs.ZShardError):
            zs.muon_scalars_bytes(zs.MuonConfig(lr=0.01, grad_scale=scale))
    zs.muon_scalars_bytes(zs.MuonConfig(lr=0.01, grad_scale=1e-45))     # a subnormal one is held


def test_a_momentum_that_is_one_in_binary32_is_refused():
    """Beside 1 - momentum, formed in binary64, it would never forget a gradient."""
    for momentum in (1.0 - 2.0 ** -26, 1.0 - 2.0 ** -53):
        with pytest.raises(zs.ZShardError):
            zs.muon_scalars_bytes(zs.MuonConfig(lr=0.01, momentum=momentum))
    sc = M.MuonScalars.from_buffer_copy(zs.muon_scalars_bytes(zs.MuonConfig(lr=0.01, momentum=1.0 - 2.0 ** -24)))
    assert sc.momentum == 1.0 - 2.0 ** -24 and sc.one_minus_momentum == 2.0 ** -24


def test_lists_refuse_tensors_of_another_device(monkeypatch):
    """A list made while one GPU was current, given tensors while another one is: a call on the
    first would follow addresses of the second.  (Two kinds of device stand for two GPUs.)"""
    monkeypatch.setattr(T, "_pointers", lambda ts, *a, **k: ([FAKE] * len(ts), ts[0].dtype if ts else None))
    x, other = torch.zeros(4, 8), torch.zeros(4, 8, device="meta")
    muon_list, mixed, grads = zs.MuonMatrices([x], [x], [x]), zs.MixedTensors([x]), zs.GradTensors([x])
    for call in (lambda: muon_list.set_grads([other]), lambda: mixed.set([other]), lambda: grads.set_grads([other]),
                 lambda: zs.ProductMatrices([x], [torch.zeros(8, 4, device="meta")], [torch.zeros(4, 4)]),
                 lambda: zs.OrthogonalizeMatrices([x], [other])):
        with pytest.raises(ValueError, match="the list on"):
            call()
    for lst in (muon_list, mixed, grads):
        assert all(t.device == x.device for ts in lst.tensors.values() for t in ts)


def test_the_side_of_a_square_matrixs_gram(monkeypatch):
    monkeypatch.setattr(T, "_pointers", lambda ts, *a, **k: ([FAKE] * len(ts), ts[0].dtype if ts else None))
    square, wide, stack, d4, d8 = (torch.zeros(s) for s in ((4, 4), (4, 8), (3, 4, 4), (4, 4), (8, 8)))

    def turned(a, d, **kw):
        return list(zs.GramMatrices(a, d, **kw).array["transposed"])
    assert turned([square, wide, wide], [d4, d4, d8]) == [0, 0, 1]
    assert turned([square], [d4], transposed=True) == [1] and turned([square], [d4], transposed=False) == [0]
    assert turned([square, wide, stack], [d4, d8, torch.zeros(3, 4, 4)], transposed=[True, None, True]) == [1, 1, 1, 1, 1]
    for a, d, kw in (([wide], [d4], True), ([wide], [d8], False), ([square], [d4], [True, False]), ([square, wide], [d4, d4], True)):
        with pytest.raises(ValueError):
            zs.GramMatrices(a, d, transposed=kw)
