"""Build libzshard.so (the library) and libzsceiling.so (the benchmark's
bandwidth-ceiling kernel, not part of the library's interface) in-tree with
hipcc for gfx950.

    python -m fsdp_sharded_optimizer_amd.build

Flags that matter for the numerics and for gfx950:
  -ffp-contract=off                          no a*b+c fusion: one rounding per operation
  -fhip-fp32-correctly-rounded-divide-sqrt   IEEE fp32 division and square root
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                             no packed-fp32 (v_pk_*_f32) instructions
  -fvisibility=hidden                        export only the C ABI (ZS_API in zshard.h)
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libzshard.so")
OBJECTS = os.path.join(HERE, "_build")
CEILING_LIB = os.path.join(HERE, "libzsceiling.so")
INCLUDE = os.path.join(ROOT, "include")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def sources(sub: str = "csrc"):
    return sorted(glob.glob(os.path.join(HERE, sub, "*.hip")))


# The calls over lists of tensors and matrices.  They are compiled into objects of their own
# first: the compiler's id of a code object depends on how many sources share
# its command, and the measured traffic of the flat step's kernels is recorded
# under the digests of their code objects.
OWN_OBJECTS = ("adamw_tensors.hip", "api_clip.hip", "api_matrices.hip", "api_tensors.hip", "clip.hip", "muon.hip",
               "norm_tensors.hip", "products.hip", "q8.hip")


def build(verbose: bool = False) -> str:
    _compile(CEILING_LIB, sources("ceiling"), verbose)
    own = [p for p in sources() if os.path.basename(p) in OWN_OBJECTS]
    os.makedirs(OBJECTS, exist_ok=True)
    objects = [os.path.join(OBJECTS, os.path.basename(p)[:-len(".hip")] + ".o") for p in own]
    flags = [f for f in FLAGS if f != "-shared"]
    with ThreadPoolExecutor(len(own)) as pool:
        list(pool.map(lambda po: _hipcc([*flags, "-I", INCLUDE, "-c", po[0], "-o", po[1]], verbose),
                      zip(own, objects)))
    return _compile(LIB, objects + [p for p in sources() if p not in own], verbose)


def _compile(lib: str, inputs, verbose: bool) -> str:
    tmp = lib + ".tmp"
    _hipcc([*FLAGS, "-I", INCLUDE, "-o", tmp, *inputs], verbose)
    os.replace(tmp, lib)
    return lib


def _hipcc(args, verbose: bool) -> None:
    cmd = [os.environ.get("HIPCC", "/opt/rocm/bin/hipcc"), *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 target feature and says so
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in proc.stderr.splitlines() if noise not in l and "(ignoring feature)" not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"hipcc failed ({proc.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


if __name__ == "__main__":
    print(build(verbose=True))
