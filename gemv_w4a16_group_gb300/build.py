"""Build the C-ABI shared library in-tree with nvcc for sm_103a (GB300).

    python -m gemv_w4a16_group_gb300.build          # incremental
    python -m gemv_w4a16_group_gb300.build --force  # full rebuild

Objects go to ``gemv_w4a16_group_gb300/_build/`` and the library to
``gemv_w4a16_group_gb300/_lib/libw4a16_gb300.so`` (both git-ignored). Each ``.cu`` is
compiled in parallel, then linked with the static CUDA runtime so the library needs
nothing but the driver at run time.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libw4a16_gb300.so")

SOURCES = ["api.cu", "quant_pack.cu", "gemv.cu", "q4b32.cu", "q4b32_mma.cu", "gemm_tc.cu",
           "no_alloc.cu", "host_cache.cu", "skinny.cu", "w8a16.cu",
           "nvfp4.cu", "fp4_mma.cu", "fp4_matmul.cu", "prepared.cu", "w8a16_mma.cu",
           "kv4_api.cu", "kv4_cache.cu", "kv4_attention.cu", "kv4_prompt.cu",
           "kv4_evict.cu"]
HEADERS = ["common.cuh", "fp4_common.cuh", "launch.h", "kv4.h", "kv4_prompt.h",
           "kv4_common.cuh"]
PUBLIC_HEADERS = ["w4a16.h", "w4a16_testing.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _newest_input() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files += [os.path.join(INCLUDE, f) for f in PUBLIC_HEADERS]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc(), *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.append("-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if it is missing or older than its sources."""
    if not force and os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= _newest_input():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
