"""Build the HIP library (libtopk_mi355x.so) in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtopk_mi355x.so")
SOURCES = ["topk_kernels.hip", "topk_linear.hip", "topk_sparse.hip", "topk_norm.hip", "topk_plan.cpp",
           "topk_abi.cpp", "topk_ops_abi.cpp"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# -amdgpu-kernarg-preload-count: the first 14 argument words of every kernel
# arrive in scalar registers with the launch instead of being loaded from the
# argument block (the kernels order their arguments for it).
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-mllvm", "-amdgpu-kernarg-preload-count=16",
         "-Wall", "-Wno-unused-function"]


def _run(cmd) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)
    return res.stderr


def build(verbose: bool = False) -> str:
    """Compile every source (in parallel, each to an object of its own) and link."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as work:
        objs = [os.path.join(work, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
            logs = list(pool.map(_run, [[HIPCC, *FLAGS, "-c", "-o", o, os.path.join(CSRC, s)]
                                        for s, o in zip(SOURCES, objs)]))
        logs.append(_run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]))
    if verbose:
        print("".join(logs))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
