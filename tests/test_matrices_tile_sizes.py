"""The shapes that tests name for a tile size take it (CPU): what a size's kernels do is
tested only where they run."""
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

from tests import matrices_tiles as tiles

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_shape_takes_the_tiles_that_it_is_named_for():
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    if torch.cuda.device_count() > 0:
        pytest.skip("host-only check: run where no GPU is visible")
    asked, want = [], []
    for dtype in (0, 1):
        for (m, n, k), side in tiles.PRODUCTS:
            asked.append(f"product {dtype} {m} {n} {k} 1")
            want.append([side])
        for (m, k), side in tiles.GRAMS:
            asked.append(f"gram {dtype} {m} 0 {k} 1")
            want.append([side])
    for (rows, cols, count), square, wide in tiles.STEPS:
        asked.append(f"muon {rows} {cols} {count}")
        want.append([square, square, wide, wide])
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "tile_sizes_driver")
        subprocess.run([hipcc, "--offload-arch=gfx950", "-O1", "-std=c++17", "-x", "hip", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", "-I", os.path.join(os.path.dirname(HERE), "include"), "-o", exe,
                        os.path.join(HERE, "sanitize", "tile_sizes_driver.cpp")], check=True, capture_output=True, text=True)
        proc = subprocess.run([exe], input="\n".join(asked) + "\n", capture_output=True, text=True, timeout=120)
    assert proc.returncode == 0, proc.stderr
    got = [[int(x) for x in line.split()] for line in proc.stdout.splitlines()]
    # (a launch without workgroups is not made: nothing of these lists has a short side up to 64)
    assert dict(zip(asked, got)) == dict(zip(asked, want))
