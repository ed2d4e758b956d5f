"""The host side of the calls over lists of tensors under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): validation, the overlap check, the tables."""
import os
import shutil
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_lists_are_clean_under_asan_and_ubsan():
    import torch
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    if torch.cuda.device_count() > 0:
        pytest.skip("host-only check: run where no GPU is visible")
    root = os.path.dirname(HERE)
    csrc = os.path.join(root, "fsdp_sharded_optimizer_amd", "csrc")
    srcs = sorted(os.path.join(csrc, f) for f in os.listdir(csrc) if f.endswith(".hip"))
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "tensors_driver")
        cmd = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-ffp-contract=off",
               "-fhip-fp32-correctly-rounded-divide-sqrt", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
               "-Xarch_host", "-fno-sanitize-recover=all", "-I", os.path.join(root, "include"), "-o", exe,
               os.path.join(HERE, "sanitize", "tensors_driver.cpp"), *srcs]
        subprocess.run(cmd, check=True, capture_output=True, text=True)
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
        proc = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
        assert proc.returncode == 0, (proc.stdout + proc.stderr)[-4000:]
        assert "runtime error" not in proc.stderr and "AddressSanitizer" not in proc.stderr, proc.stderr[-4000:]
        assert "tensors sanitizer drive: ok" in proc.stdout
