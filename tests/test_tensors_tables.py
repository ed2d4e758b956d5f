"""The launch tables of the calls over lists of tensors, looked up on the host as
the kernels look them up: every element of every tensor is taken once, in order,
at its address (CPU, under AddressSanitizer and UndefinedBehaviorSanitizer)."""
import os
import shutil
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_tables_cover_every_list():
    import torch
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    if torch.cuda.device_count() > 0:
        pytest.skip("host-only check: run where no GPU is visible")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "tables_driver")
        cmd = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-x", "hip", "-Xclang", "-target-feature", "-Xclang",
               "-packed-fp32-ops", "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
               "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all", "-I",
               os.path.join(os.path.dirname(HERE), "include"), "-o", exe, os.path.join(HERE, "sanitize", "tables_driver.cpp")]
        subprocess.run(cmd, check=True, capture_output=True, text=True)
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
        proc = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
        assert proc.returncode == 0 and "tables: ok" in proc.stdout, (proc.stdout + proc.stderr)[-4000:]
