"""Build the CUDA library libms_b200.so in-tree with nvcc for sm_100a, and the Python extension _paged.so
(host code against torch's headers) that calls it.

Usage: python decoder_only_transformer_int4_b200/build.py [--force] [--verbose-ptxas]
(run by path: importing the package itself loads the library this script builds)
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libms_b200.so")
SOURCES = ["k_elementwise.cu", "k_gemv.cu", "k_gemm_f16.cu", "k_w4a8.cu", "k_gemm_i8.cu", "k_attn.cu", "k_attn_tc.cu", "k_decode_persistent.cu", "k_cond.cu", "ms_runtime.cu",
           "ms_noalloc.cu", "k_paged.cu", "k_attn_paged.cu", "k_verify.cu", "ms_paged.cu"]
EXT = os.path.join(HERE, "_paged" + sysconfig.get_config_var("EXT_SUFFIX"))
EXT_SOURCE = "py_paged.cpp"
EXT_STAMP = os.path.join(BUILD, "extension")   # what it was built for
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, ptxas_v: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", os.path.join(HERE, "..", "include"), "-c",
           os.path.join(CSRC, src), "-o", obj]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if ptxas_v:
        sys.stderr.write(r.stderr)
    return obj


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps.append(os.path.join(HERE, "..", "include", "ms.h"))
    deps.append(os.path.join(CSRC, src))
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _extension_for() -> str:
    """The torch and the Python that the extension is built for."""
    return f"torch {importlib.metadata.version('torch')}, Python {sysconfig.get_config_var('EXT_SUFFIX')}"


def _extension_stale() -> bool:
    if _stale(EXT, EXT_SOURCE) or not os.path.exists(EXT_STAMP):
        return True
    with open(EXT_STAMP) as f:
        return f.read() != _extension_for()


def _build_extension() -> None:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    lib = os.path.join(torch, "lib")
    tmp = EXT + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, EXT_SOURCE), "-o", tmp, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python",
           "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{EXT_SOURCE} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    with open(EXT_STAMP, "w") as f:
        f.write(_extension_for())


def build(force: bool = False, ptxas_v: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    todo = [s for s in SOURCES if force or ptxas_v or
            _stale(os.path.join(BUILD, os.path.splitext(s)[0] + ".o"), s)]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        list(ex.map(lambda s: _compile(s, ptxas_v), todo))
    objs = [os.path.join(BUILD, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    if todo or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-ldl", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if force or _extension_stale():
        _build_extension()
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_v=a.verbose_ptxas))
