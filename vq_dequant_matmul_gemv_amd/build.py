"""Build libvqmi.so (the HIP kernels + C ABI) in-tree with hipcc for gfx950.

    python -m vq_dequant_matmul_gemv_amd.build        # or build() from Python

Sources: csrc/*.hip and csrc/*.cpp; public header: <repo>/include/vq.h.
Output: vq_dequant_matmul_gemv_amd/lib/libvqmi.so.  Always recompiles.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libvqmi.so")
OBJDIR = os.path.join(ROOT, "_build")

ARCH = "gfx950"

# Packed-fp32 VALU forms are switched off: only scalar/packed-fp16 arithmetic
# is used on purpose; hipcc's host pass warns that it does not know the
# feature, which is harmless.
# Kernel-argument preloading: the first 10 scalar arguments of a kernel (the
# GEMV's pointers, row count and row split: 14 SGPRs) arrive in SGPRs at wave
# launch.
COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Werror", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-kernarg-preload-count=10",
    "-fno-gpu-rdc", "-I", INCLUDE, "-I", CSRC,
]

# Per-source flags.  vq_fp8.hip scales every matrix product's sum into its
# accumulators with VALU instructions, which read VGPRs only: the products'
# destinations must not be AGPRs.
EXTRA = {
    "vq_fp8.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
}


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *COMMON, *EXTRA.get(os.path.basename(src), []), "-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
