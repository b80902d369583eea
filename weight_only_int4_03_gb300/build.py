"""Builds libw4a16.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file compiles to an object in parallel, then one nvcc link makes the shared
library under weight_only_int4_03_gb300/_lib/.  The CUDA runtime is linked statically, so the
library needs only the driver at run time.  Beside it comes a small extension module for the
interpreter that builds (the decode-step operators called without ctypes), where Python's headers are
installed.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libw4a16.so")
CALL_PATH = os.path.join(LIB_DIR, "_w4a16_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
INCLUDE = os.path.join(ROOT, "include")
PYTHON_INCLUDE = sysconfig.get_paths()["include"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["w4a16_gemm.cu", "w4a16_decode.cu", "w4a16_aux.cu", "w4a16_api.cu", "w4a16_noalloc.cu",
           "w4a16_loader.cu", "w4a16_rope.cu", "w4a16_attention.cu",
           "w4a16_moe_layer.cu", "w4a16_norm_rope.cu", "w4a16_kv4_attention.cu", "w4a16_sample.cu"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the W4A16 library cannot be built")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "w4a16.h"))
    return files


def _has_python_headers() -> bool:
    return os.path.exists(os.path.join(PYTHON_INCLUDE, "Python.h"))


def up_to_date() -> bool:
    outputs = [LIB_PATH, CALL_PATH] if _has_python_headers() else [LIB_PATH]
    if not all(os.path.exists(f) for f in outputs):
        return False
    t = min(os.path.getmtime(f) for f in outputs)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and return the path of libw4a16.so."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "--expt-relaxed-constexpr"]
    if ptxas_info:
        common += ["-Xptxas", "-v"]
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, "-c", os.path.join(CSRC, src), "-o", obj] + common
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, proc in procs:
        out, _ = proc.communicate()
        text = out.decode(errors="replace")
        if proc.returncode != 0:
            failed.append(f"--- {src} ---\n{text}")
        elif verbose or ptxas_info:
            sys.stdout.write(text)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"])
    os.replace(tmp, LIB_PATH)
    if _has_python_headers():
        tmp = CALL_PATH + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc, "-shared", "-cudart", "none", "-O2", "-std=c++17", "-Xcompiler", "-fPIC",
                               "-I", INCLUDE, "-I", PYTHON_INCLUDE, os.path.join(CSRC, "w4a16_call.cpp"), "-o", tmp,
                               "-L", LIB_DIR, "-lw4a16", "-Xlinker", "-rpath,$ORIGIN"])
        os.replace(tmp, CALL_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
