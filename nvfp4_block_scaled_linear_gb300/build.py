"""Build libnvfp4_linear.so (sm_103a) in-tree with nvcc.

    python -m nvfp4_block_scaled_linear_gb300.build [--force] [--verbose]

Output: nvfp4_block_scaled_linear_gb300/_build/libnvfp4_linear.so (ignored by
git), from the linear layer's translation unit (csrc/) and the attention
block's (csrc_attention/).  The CUDA runtime is linked as a shared library so
that the process shares one runtime (current device, streams) with PyTorch.
"""
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libnvfp4_linear.so")
MAIN = os.path.join(CSRC, "nvfp4_linear.cu")
CSRC_ATTENTION = os.path.join(HERE, "csrc_attention")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) +
                  glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC_ATTENTION, "*.cu")) +
                  glob.glob(os.path.join(CSRC_ATTENTION, "*.cuh")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def _units():
    """The translation units: the linear layer's and the attention block's."""
    return [MAIN] + sorted(glob.glob(os.path.join(CSRC_ATTENTION, "*.cu")))


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(s) for s in _sources())
        if os.path.getmtime(LIB) >= newest:
            return LIB
    tmp = LIB + ".tmp.%d" % os.getpid()
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    objects, jobs = [], []
    try:
        # one nvcc per translation unit, all at once
        for unit in _units():
            obj = "%s.%s.o" % (tmp, os.path.splitext(os.path.basename(unit))[0])
            objects.append(obj)
            jobs.append(subprocess.Popen([_nvcc(), *flags, "-c", "-o", obj, unit]))
        failed = [j.args for j in jobs if j.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        subprocess.run([_nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objects],
                       check=True)
    finally:
        for j in jobs:
            j.wait()
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
