"""Builds the C-ABI library ``lib/libhsdp_fsdp.so`` in-tree.

The translation units are compiled in parallel and linked with nvcc:
  * csrc/fsdp_kernels.cu -- the sm_103a kernels (nvcc, one -gencode)
  * csrc/fsdp_bulk.cu    -- the bulk-fed fused reduce of a capped grid
  * csrc/fsdp_noalloc.cu -- the allocation-free fused gradient sync
  * csrc/fsdp_embedding.cu, fsdp_dropout.cu, fsdp_norm.cu, fsdp_ffn.cu, fsdp_ortho.cu -- the
    training operators
  * csrc/fsdp_capi.cpp   -- plan, bindings and entry points (host C++)
  * csrc/fsdp_ops_capi.cpp -- entry points of the training operators (host C++)
No fast-math, no FMA contraction, no flush-to-zero: the kernels' additions,
divisions and conversions are single IEEE operations.
"""
from __future__ import annotations

import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(HERE, "lib")
LIB_NAME = "libhsdp_fsdp.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-Wall", "-ftz=false",
              "-prec-div=true", "-prec-sqrt=true", "-fmad=false", "--expt-relaxed-constexpr"]
CUDA_SOURCES = ["fsdp_kernels.cu", "fsdp_noalloc.cu", "fsdp_bulk.cu", "fsdp_embedding.cu", "fsdp_dropout.cu",
                "fsdp_norm.cu", "fsdp_ffn.cu", "fsdp_ortho.cu"]
CXX_SOURCES = ["fsdp_capi.cpp", "fsdp_ops_capi.cpp"]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra"]


def cuda_home():
    for c in [os.environ.get("CUDA_HOME"), "/usr/local/cuda"]:
        if c and os.path.exists(os.path.join(c, "bin", "nvcc")):
            return c
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(nvcc))
    raise RuntimeError("nvcc not found: set CUDA_HOME")


def library_path():
    return os.path.join(LIB_DIR, LIB_NAME)


def build(verbose: bool = False, extra_nvcc=()) -> str:
    cuda = cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    os.makedirs(LIB_DIR, exist_ok=True)
    inc = ["-I", INCLUDE, "-I", CSRC]
    tag = str(os.getpid())
    obj = {f: os.path.join(LIB_DIR, f"{os.path.splitext(f)[0]}.{tag}.o") for f in CUDA_SOURCES + CXX_SOURCES}
    jobs = [[nvcc, *ARCH, *NVCC_FLAGS, *extra_nvcc, *inc, "-c", os.path.join(CSRC, f), "-o", obj[f]]
            for f in CUDA_SOURCES]
    jobs += [["g++", *CXX_FLAGS, *inc, "-I", os.path.join(cuda, "include"), "-c", os.path.join(CSRC, f), "-o", obj[f]]
             for f in CXX_SOURCES]
    procs = [subprocess.Popen(j, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for j in jobs]
    failed = []
    for j, p in zip(jobs, procs):
        out, _ = p.communicate()
        if verbose or p.returncode:
            print(out, end="")
        if p.returncode:
            failed.append(" ".join(j))
    if failed:
        raise RuntimeError("compile failed: " + "; ".join(failed))
    tmp = os.path.join(LIB_DIR, f"{LIB_NAME}.{tag}")
    subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "shared", *obj.values(), "-o", tmp,
                    "-Xlinker", "-rpath," + os.path.join(cuda, "lib64")], check=True)
    os.replace(tmp, library_path())
    for o in obj.values():
        os.remove(o)
    return library_path()


if __name__ == "__main__":
    print(build(verbose=True))
