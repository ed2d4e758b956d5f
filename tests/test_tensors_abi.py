"""The calls over lists of tensors on the host: exports, sizes and refusals.

No call reaches a launch (there is no GPU here): each fails validation or has
nothing to do.  Pointers passed are never dereferenced.
"""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

import fsdp_sharded_optimizer_amd as zs
from fsdp_sharded_optimizer_amd import _binding as B
from fsdp_sharded_optimizer_amd import tensors as T
from tests import tensors_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
MIB = 1 << 20


@pytest.fixture(autouse=True)
def no_launch_reached():
    yield
    assert zs.lib().zs_last_hip_error() == 0, "a call got past validation to a kernel launch"


L = T._lib()
HP = B.AdamW(3e-4, 0.9, 0.95, 1e-8, 0.1, 1.0 / 64, 1.0, 0.0, 3)
hp = ctypes.byref(HP)


def hp_with(**kw):
    h = B.AdamW(3e-4, 0.9, 0.95, 1e-8, 0.1, 1.0 / 64, 1.0, 0.0, 3)
    for k, v in kw.items():
        setattr(h, k, v)
    return ctypes.byref(h)


def fill(struct, rows):
    a = (struct * max(len(rows), 1))()
    for k, row in enumerate(rows):
        for name, value in zip((f for f, _ in struct._fields_), row):
            setattr(a[k], name, value)
    return a


def test_exports_match_the_header():
    text = open(os.path.join(ROOT, "include", "zshard_tensors.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*ZS_API\s+(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", text, flags=re.M))
    assert names == set(zs.TENSOR_EXPORTS)
    for name in names:
        assert getattr(L, name) is not None


def test_header_is_plain_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src = tmp_path / "c.c"
    src.write_text('#include "zshard_tensors.h"\n#include <stdio.h>\nint main(void) {\n'
                   "  zs_adamw_q8_scalars sc; zs_adamw hp = {.lr = 1e-3, .beta1 = 0.9, .beta2 = 0.95, .eps = 1e-8,"
                   " .grad_scale = 1.0, .step = 1};\n"
                   "  if (adamw_q8_scalars(&hp, 7u, &sc) != ZS_OK || sc.reserved != 0) return 1;\n"
                   "  if (adamw_step_tensors(&hp, NULL, 0, ZS_F32, ZS_BF16, NULL, NULL) != ZS_OK) return 2;\n"
                   '  printf("%lld\\n", (long long)moments_q8_bytes(1000000));\n  return 0;\n}\n')
    exe = str(tmp_path / "c")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Wextra", "-Wpedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-o", exe, str(src), B.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(B.LIB_PATH)}"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and int(out.stdout) == zs.moments_q8_bytes(10**6)


def test_moments_q8_bytes():
    for n in (0, 1, 2, 255, 256, 257, 1023, 1024, 1025, 10**6, 842_301_952, 1 << 39):
        b = zs.moments_q8_bytes(n)
        assert b % 128 == 0 and b >= 2 * n + 2 * -(-n // zs.Q8_BLOCK) and b <= 2.0079 * n + 2176
    for n in (-1, (1 << 39) + 1):
        assert L.moments_q8_bytes(n) == -1
        with pytest.raises(ValueError):
            zs.moments_q8_bytes(n)


def test_workspace_bytes():
    def need(numels, dtype):
        return L.grad_norm_sq_tensors_workspace_bytes(fill(B.Tensor, [(0, n) for n in numels]), len(numels), dtype)
    assert need([], 0) == 0 and need([0, 0], 1) == 0
    assert need([1, 0, 4096], 0) == 16 and need([4097], 0) == 16 and need([4097], 1) == 8
    assert need([1] * 3000, 0) == (3000 + 2048) * 8
    assert need([-1], 0) == -1 and need([1 << 39, 1], 0) == -1 and need([5], 2) == -1
    assert L.grad_norm_sq_tensors_workspace_bytes(None, 1, 0) == -1
    assert L.grad_norm_sq_tensors_workspace_bytes(None, -1, 0) == -1


def test_q8_scalars_are_the_steps_scalars_and_the_key():
    for step, seed in ((1, 0), (3, 5), (1000, 0xFFFFFFFF), ((1 << 32) + 9, 12)):
        cfg = zs.AdamWConfig(lr=3e-4, beta2=0.95, weight_decay=0.1, step=step)
        raw = zs.q8_scalars_bytes(cfg, seed)
        assert raw[:56] == zs.scalars_bytes(cfg)
        assert int.from_bytes(raw[56:60], "little") == ref.key_of(seed, step) and raw[60:] == bytes(4)
    assert L.adamw_q8_scalars(hp, 0, None) == B.ZS_EINVAL
    assert L.adamw_q8_scalars(hp_with(step=0), 0, ctypes.byref(T.AdamWQ8Scalars())) == B.ZS_EINVAL
    with pytest.raises(ValueError):
        zs.q8_scalars_bytes(zs.AdamWConfig(lr=1e-3), 1 << 32)
    with pytest.raises(ValueError):
        zs.q8_scalars_bytes(zs.AdamWConfig(lr=1e-3), -1)


BAD_HP = [dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(lr=float("inf")),
          dict(weight_decay=-1.0), dict(grad_scale=0.0), dict(max_norm=float("nan")), dict(extra_norm_sq=-1.0)]


def step_rows(n=1000, tensors=2):
    """Disjoint buffers, 1 MiB apart: (param, grad, exp_avg, exp_avg_sq, copy, numel)."""
    return [[FAKE + (5 * k + j) * MIB for j in range(4)] + [FAKE + (5 * k + 4) * MIB, n] for k in range(tensors)]


def step(rows, h=hp, count=None, pd=0, gd=0, norm=None):
    return L.adamw_step_tensors(h, fill(T.AdamWTensor, rows), len(rows) if count is None else count, pd, gd, norm, None)


def step_dev(rows, sc, pd=0, gd=0, norm=None):
    return L.adamw_step_tensors_dev(sc, fill(T.AdamWTensor, rows), len(rows), pd, gd, norm, None)


def q8_rows(n=1000, tensors=2):
    return [[FAKE + (4 * k + j) * MIB for j in range(4)] + [n] for k in range(tensors)]


def step_q8(rows, h=hp, count=None, pd=0, gd=0, norm=None):
    return L.adamw_step_tensors_q8(h, 0, fill(T.AdamWQ8Tensor, rows), len(rows) if count is None else count, pd, gd,
                                   norm, None)


def step_q8_dev(rows, sc, pd=0, gd=0, norm=None):
    return L.adamw_step_tensors_q8_dev(sc, fill(T.AdamWQ8Tensor, rows), len(rows), pd, gd, norm, None)


def edited(rows, k, j, value):
    rows = [list(r) for r in rows]
    rows[k][j] = value
    return rows


@pytest.mark.parametrize("call,dev,rows,state", [(step, step_dev, step_rows, (2, 3)), (step_q8, step_q8_dev, q8_rows, (2,))])
def test_steps_reject(call, dev, rows, state):
    good = rows()
    assert call([]) == B.ZS_OK and call(rows(0)) == B.ZS_OK
    assert call([[0] * (len(good[0]) - 1) + [0]]) == B.ZS_OK          # an empty tensor's pointers are not looked at
    for bad in BAD_HP:
        assert call(good, h=hp_with(**bad)) == B.ZS_EINVAL, bad
    assert call(good, h=None) == B.ZS_EINVAL
    assert call(good, count=-1) == B.ZS_EINVAL
    assert call(good, pd=2) == B.ZS_EINVAL and call(good, gd=-1) == B.ZS_EINVAL
    assert call(good, norm=FAKE - 4) == B.ZS_EINVAL
    assert dev(good, FAKE - 60) == B.ZS_EINVAL and dev(good, None) == B.ZS_EINVAL
    last = len(good[0]) - 1
    copy = last - 1
    for j in range(copy):
        assert call(edited(good, 1, j, 0)) == B.ZS_EINVAL, j          # null
    for j in range(2):
        assert call(edited(good, 1, j, good[1][j] + 2)) == B.ZS_EINVAL, j      # fp32 off 4 bytes
        no_copy = [r[:copy] + [0, r[last]] for r in good]
        assert call(edited(no_copy, 1, j, good[1][j] + 1), pd=1, gd=1) == B.ZS_EINVAL, j
    for j in state:
        assert call(edited(good, 1, j, good[1][j] + 2)) == B.ZS_EINVAL, j
    assert call(edited(good, 1, copy, good[1][copy] + 1)) == B.ZS_EINVAL
    assert call(good, pd=1) == B.ZS_EINVAL                            # a re-cast of bf16 parameters
    assert call(edited(good, 1, last, -5)) == B.ZS_EINVAL
    assert call(edited(good, 1, last, (1 << 39) + 1)) == B.ZS_EINVAL
    assert call(edited(edited(good, 0, last, 1 << 39), 1, last, 1)) == B.ZS_EINVAL
    # overlaps: each pair of one tensor's buffers, across tensors, the norm and the scalars
    for a in range(copy + 1):
        for b in range(a):
            assert call(edited(good, 0, a, good[0][b] + 16)) == B.ZS_EOVERLAP, (a, b)
            assert call(edited(good, 1, a, good[0][b] + 16)) == (B.ZS_EOVERLAP), (a, b)
        if a != 1:
            assert call(good, norm=good[1][a] + 8) == B.ZS_EOVERLAP
            assert dev(good, good[1][a] + 8) == B.ZS_EOVERLAP
    assert call(edited(good, 1, 0, good[0][0])) == B.ZS_EOVERLAP      # the same parameter twice


def test_q8_state_alignment():
    good = q8_rows()
    assert step_q8(edited(good, 0, 2, good[0][2] + 8)) == B.ZS_EINVAL
    rows = [[FAKE, FAKE + MIB, FAKE + 2 * MIB + 8, 100]]
    a = fill(T.MomentsQ8, rows)
    assert L.moments_q8_encode(a, 1, 0, 0, None) == B.ZS_EINVAL and L.moments_q8_decode(a, 1, 0, None) == B.ZS_EINVAL


def test_conversions_reject():
    good = [[FAKE + (3 * k + j) * MIB for j in range(3)] + [1000] for k in range(2)]
    for f in (lambda a, n, d: L.moments_q8_encode(a, n, d, 0, None), lambda a, n, d: L.moments_q8_decode(a, n, d, None)):
        assert f(None, 0, 0) == B.ZS_OK and f(fill(T.MomentsQ8, [[0, 0, 0, 0]]), 1, 0) == B.ZS_OK
        assert f(None, 1, 0) == B.ZS_EINVAL and f(fill(T.MomentsQ8, good), -1, 0) == B.ZS_EINVAL
        assert f(fill(T.MomentsQ8, good), 2, 2) == B.ZS_EINVAL
        assert f(fill(T.MomentsQ8, edited(good, 1, 2, 0)), 2, 0) == B.ZS_EINVAL
        assert f(fill(T.MomentsQ8, edited(good, 1, 0, good[1][0] + 2)), 2, 0) == B.ZS_EINVAL
        assert f(fill(T.MomentsQ8, edited(good, 1, 1, good[1][1] + 1)), 2, 1) == B.ZS_EINVAL
        assert f(fill(T.MomentsQ8, edited(good, 1, 3, -1)), 2, 1) == B.ZS_EINVAL
        for a in (0, 1):
            assert f(fill(T.MomentsQ8, edited(good, 1, a, good[0][2] + 512)), 2, 0) == B.ZS_EOVERLAP
    # two states into one buffer; two values into one place (two reads of it may alias: not a launch here)
    assert L.moments_q8_encode(fill(T.MomentsQ8, edited(good, 1, 2, good[0][2])), 2, 0, 0, None) == B.ZS_EOVERLAP
    assert L.moments_q8_decode(fill(T.MomentsQ8, edited(good, 1, 1, good[0][0])), 2, 0, None) == B.ZS_EOVERLAP
    # neither destination: nothing to do
    assert L.moments_q8_decode(fill(T.MomentsQ8, [[0, 0, FAKE, 1000]]), 1, 0, None) == B.ZS_OK


def test_norm_rejects():
    good = [[FAKE, 5000], [FAKE + MIB, 300]]
    out, ws = FAKE + 2 * MIB, FAKE + 3 * MIB

    def f(rows, count=None, d=0, scale=1.0, o=out, w=ws, nbytes=MIB):
        return L.grad_norm_sq_tensors(fill(B.Tensor, rows), len(rows) if count is None else count, d, scale, o, w,
                                      nbytes, None)
    assert f(good, count=-1) == B.ZS_EINVAL and f(good, d=3) == B.ZS_EINVAL
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert f(good, scale=scale) == B.ZS_EINVAL
    assert f(good, o=None) == B.ZS_EINVAL and f(good, o=out + 4) == B.ZS_EINVAL
    assert f(good, w=None) == B.ZS_EINVAL and f(good, w=ws + 4) == B.ZS_EINVAL
    assert f(good, nbytes=23) == B.ZS_EWORKSPACE and f(good, nbytes=-1) == B.ZS_EWORKSPACE
    assert f(edited(good, 1, 0, 0)) == B.ZS_EINVAL and f(edited(good, 1, 0, FAKE + MIB + 2)) == B.ZS_EINVAL
    assert f(edited(good, 1, 0, FAKE + MIB + 1), d=1) == B.ZS_EINVAL
    assert f(edited(good, 1, 1, -1)) == B.ZS_EINVAL
    assert f(good, o=FAKE + 80) == B.ZS_EOVERLAP and f(good, w=FAKE + 80) == B.ZS_EOVERLAP
    assert f(good, w=out) == B.ZS_EOVERLAP
    assert L.grad_norm_sq_tensors(None, 1, 0, 1.0, out, ws, MIB, None) == B.ZS_EINVAL


def test_overlaps_are_found_in_any_order():
    """Random lists of small buffers against the pairwise rule: a written buffer
    shares no byte with any other.  Only lists with an overlap are passed (no
    call may reach a launch)."""
    rng = random.Random(11)
    seen = 0
    for _ in range(3000):
        count = rng.choice([1, 2, 3, 8, 150])
        span = count * rng.choice([4, 40, 4000])
        rows, spans = [], []
        for _ in range(count):
            n = rng.randrange(0, 20)
            at = [FAKE + 4 * rng.randrange(span) for _ in range(4)] + [FAKE + 2 * rng.randrange(2 * span)]
            if rng.random() < 0.3:
                at[4] = 0
            rows.append(at + [n])
            if n:
                spans += [(p, p + n * sz, j != 1) for j, (p, sz) in enumerate(zip(at, (4, 4, 4, 4, 2))) if p]
        hit = any(a[0] < b[1] and b[0] < a[1] and (a[2] or b[2])
                  for i, a in enumerate(spans) for b in spans[:i])
        if hit:
            seen += 1
            assert step(rows) == B.ZS_EOVERLAP
    assert seen > 1000


def test_lists_refuse_what_cannot_be_marshalled():
    x = torch.zeros(4)
    for make in (lambda: zs.GradTensors([x]), lambda: zs.AdamWTensors([x], [x], [x], [x]),
                 lambda: zs.AdamWQ8Tensors([x], [x], [x]), lambda: zs.Q8Moments([x.to(torch.uint8)], [x], [x])):
        with pytest.raises(ValueError, match="GPU tensor"):
            make()
    with pytest.raises(TypeError):
        zs.GradTensors([None])
    with pytest.raises(ValueError):
        zs.AdamWTensors([], [x], [], [])
    with pytest.raises(ValueError):
        zs.Q8Moments([x], None, None)
    with pytest.raises(ValueError):
        zs.Q8Moments([], [x], [])


def test_a_missing_library_is_an_error(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libzshard.so"))
    with pytest.raises(RuntimeError):
        zs.moments_q8_bytes(5)


def test_gradients_of_another_device_are_refused():
    """Marshalled while another GPU was current: the check is of the lists'
    devices, so descriptors without tensors behind them do."""
    def of(cls, struct, index):
        lst = object.__new__(cls)
        T._List.__init__(lst, struct, [4, 0], torch.device("cuda", index))
        return lst
    for cls, struct in ((T.AdamWTensors, T.AdamWTensor), (T.AdamWQ8Tensors, T.AdamWQ8Tensor)):
        lst, here, there = of(cls, struct, 0), of(T.GradTensors, B.Tensor, 0), of(T.GradTensors, B.Tensor, 1)
        for k, g in enumerate((here, there)):
            g._set("ptr", [None, None], [FAKE + k, 0])
            g.grad_dtype = B.ZS_F32
        lst.set_grads(here)
        with pytest.raises(ValueError, match="cuda:1"):
            lst.set_grads(there)
        assert list(lst.array["grad"]) == [FAKE, 0]      # the refused ones changed nothing
