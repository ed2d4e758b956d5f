"""The kernels' look-up of a workgroup's tile, the library's own functions, on the
tables that the calls over lists of tensors fill (CPU, under AddressSanitizer and
UndefinedBehaviorSanitizer): every tile of every tensor is taken once, in the plain
order and in the runs of lists off cache lines."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_tile_is_taken_once(tmp_path):
    import torch
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    if torch.cuda.device_count() > 0:
        pytest.skip("host-only check: run where no GPU is visible")
    exe = str(tmp_path / "lookup_driver")
    cmd = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-x", "hip", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
           "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all", "-I",
           os.path.join(os.path.dirname(HERE), "include"), "-o", exe, os.path.join(HERE, "sanitize", "lookup_driver.cpp")]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    proc = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert proc.returncode == 0 and "look-up: ok" in proc.stdout, (proc.stdout + proc.stderr)[-4000:]
