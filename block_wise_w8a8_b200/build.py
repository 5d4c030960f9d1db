"""Build libw8a8.so (the C-ABI library) in-tree with nvcc for sm_100a."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "w8a8.cu")
DEPS = [os.path.join(HERE, "csrc", f) for f in ("w8a8.cu", "block_norm.cuh", "common.cuh", "fp4.cuh", "fp4_gemm.cuh", "fp4_host.cuh",
                                               "gemm.cuh", "norm.cuh", "quant.cuh")] + \
    [os.path.join(ROOT, "include", "w8a8.h")]
LIB = os.path.join(HERE, "libw8a8.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-Xcompiler", "-Wall", "-cudart", "static"]


def stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in DEPS)


def build(force=False, verbose_ptxas=False):
    if not force and not stale():
        return LIB
    cmd = [NVCC, *FLAGS, SRC, "-o", LIB]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    subprocess.run(cmd, check=True)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose_ptxas="-v" in sys.argv)
    print(LIB)
