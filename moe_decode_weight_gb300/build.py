"""Compile the CUDA sources under ``csrc/`` into the in-tree shared library ``libmdw.so``.

sm_103a only (GB300): ``nvcc -gencode arch=compute_103a,code=sm_103a``. Each translation
unit is compiled in parallel, then linked with the CUDA runtime statically.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmdw.so")
BINDING = os.path.join(PKG, "_binding.so")            # CPython extension: argument marshalling (csrc/binding.c)
TRACE_LIB = os.path.join(PKG, "libmdw_trace.so")     # profiling build (-DMDW_TRACE), never loaded by the API
SOURCES = ["moe.cu", "lm_head.cu", "abi.cu", "noalloc.cu", "sampler.cu", "w4_linear.cu", "w4_tensor.cu",
           "kv_cache.cu", "tree_attention.cu", "tree_attention_rows.cu"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=default",
         "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libmdw.so")
    return path


def _compile(src: str, trace: bool = False) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + (".trace.o" if trace else ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, *(["-DMDW_TRACE"] if trace else []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _binding() -> None:
    """The extension is not needed for the C library or the decode step's calls: without a C compiler or
    Python's headers a warning says so, and the calls that want it raise."""
    tmp = BINDING + ".tmp"
    cc, headers = shutil.which("gcc") or shutil.which("cc"), sysconfig.get_paths()["include"]
    if cc is None or not os.path.exists(os.path.join(headers, "Python.h")):
        if os.path.exists(BINDING):
            os.remove(BINDING)                        # an earlier build's may not match the library
        warnings.warn(f"no C compiler or no Python.h in {headers}: {os.path.basename(BINDING)} is not built, "
                      "and the attention sub-layer's calls from Python are not available")
        return
    cmd = [cc, "-O2", "-std=c11", "-Wall", "-shared", "-fPIC", "-I" + headers,
           "-I" + INCLUDE, os.path.join(CSRC, "binding.c"), "-o", tmp, "-lm"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on binding.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False, trace: bool = False) -> str:
    """Build libmdw.so and _binding.so (always rebuilds); returns the library's path. trace=True builds the profiling
    library libmdw_trace.so instead: the same kernels with %globaltimer stamps at their phase
    boundaries (read by moe_decode_weight_gb300.phase_trace); the product library is untouched."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda src: _compile(src, trace), SOURCES))
    out = TRACE_LIB if trace else LIB
    tmp = out + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    if not trace:
        _binding()
    if verbose:
        print(f"built {out}")
    return out


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
