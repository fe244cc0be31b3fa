"""Build libmxq.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a.

    python -m mxfp_block_scaled_b200.build [--force]
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmxq.so")
SOURCES = ["api.cu", "nvfp4.cu", "weighted.cu", "mx.cu", "verify.cu", "noalloc.cu",
           "fp8.cu", "gemm.cu", "moe.cu", "linear.cu", "cache.cu", "attention.cu",
           "attention_rows.cu", "attention_tiles.cu"]
HEADERS = ["mxq_device.cuh", "mxq_internal.h", "mxq_layer.h", "mxq_tma.cuh", "mxq_tcgen05.cuh", "mxq_mma.cuh",
           "mxq_cache.cuh", "mxq_cluster.cuh", "attention.cuh",
           "nvfp4_block.cuh", "mx_block.cuh"]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
# No --use_fast_math: denormals are kept and every division / reciprocal
# that decides a code is an IEEE round-to-nearest operation.
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files += [os.path.join(INCLUDE, f) for f in ("mxq.h", "mxq_test.h")]
    return files


def needs_build():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force=False, verbose=False):
    if not force and not needs_build():
        return LIB
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for s in SOURCES:
        obj = os.path.join(objdir, s.replace(".cu", ".o"))
        cmd = [NVCC, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", obj]
        if verbose:
            print(" ".join(cmd))
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    # -z defs: an unresolved symbol fails the link instead of the first dlopen
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xlinker", "-z,defs",
           "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
