"""In-tree build of libflce.so (the C-ABI library) for sm_103a, and of _flce_ops.so, the
Python extension that makes the ordinary calls of include/flce_ops.h.

Each .cu translation unit is compiled in parallel with nvcc and linked into
linear_cross_entropy_flce_gb300/libflce.so. No cmake; CUDA's runtime is linked
statically, and the driver's tensor-map encoder is looked up at run time, so the
library loads on a machine without a GPU driver.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libflce.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]

SOURCES = ["flce_api.cu", "flce_reduce.cu", "flce_gemm_lse.cu", "flce_gemm_grad.cu",
           "flce_gemm_f32.cu", "flce_gemm_logp.cu", "flce_gemm_few.cu",
           "flce_noalloc.cu", "flce_ce.cu",
           "flce_ops_api.cu", "flce_logprobs.cu", "flce_logprob_merge.cu", "flce_norm.cu",
           "flce_norm_stream.cu", "flce_norm_stream_grad.cu",
           "flce_clip.cu"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


EXT = os.path.join(PKG, "_flce_ops.so")


def _compile_ext() -> str:
    """Compile py_ops.cpp against the installed PyTorch's headers (not imported for it)."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    obj = os.path.join(BUILD, "py_ops.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC",
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(torch, "include"),
           "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), "-c", os.path.join(CSRC, "py_ops.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for py_ops.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_ext(obj: str) -> None:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    tmp = EXT + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libflce.so",
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,--no-as-needed"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _flce_ops.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def _finish_ext(obj) -> None:
    """Link _flce_ops.so from its object (a future). Where it cannot be built, without PyTorch's
    headers for one, the package makes every call through libflce.so alone: said, not raised."""
    try:
        _link_ext(obj.result())
    except Exception as e:
        if os.path.exists(EXT):   # of other sources than libflce.so's
            os.remove(EXT)
        warnings.warn(f"built without _flce_ops.so, calls take longer on the host: {e}", RuntimeWarning)


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libflce.so (whose path is returned) and _flce_ops.so."""
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext_obj = ex.submit(_compile_ext)
        logs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    if verbose or ptxas_info:
        for s, log in zip(SOURCES, logs):
            if log.strip():
                print(f"--- {s}\n{log}", file=sys.stderr)
    objs = [os.path.join(BUILD, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-Xlinker", "--no-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _finish_ext(ext_obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
