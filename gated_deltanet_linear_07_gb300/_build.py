"""Builds libgdn_gb300.so in-tree with nvcc for sm_103a (one translation unit
per .cu file, compiled in parallel, linked with -shared).  No cmake, no torch
extension machinery: the library is a plain C ABI over the CUDA runtime.  Beside
it goes a small CPython module that marshals the attention calls (gcc and the
interpreter's headers)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libgdn_gb300.so")
CALLS_SRC = os.path.join(CSRC, "attn_calls.c")       # the attention calls' marshalling
# by the interpreter's tag: a module built for one is none for another
CALLS = os.path.join(PKG, "_attn_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-Xptxas", "-v", "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgdn_gb300.so")
    return cand


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".c"))]
    out.append(os.path.join(ROOT, "include", "gdn.h"))
    return out


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(p) <= t for p in _deps() + [__file__])


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs, logs = [], {}

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr[-6000:]}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        for obj, log in ex.map(compile_one, sources()):
            objs.append(obj)
            logs[obj] = log
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        for obj, log in logs.items():
            f.write(f"== {os.path.basename(obj)}\n{log}\n")
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)
    tmp = CALLS + f".tmp{os.getpid()}"
    r = subprocess.run(["gcc", "-O2", "-std=c99", "-Wall", "-Werror", "-shared", "-fPIC",
                        "-fvisibility=hidden", "-I", sysconfig.get_paths()["include"],
                        "-I", os.path.join(ROOT, "include"), CALLS_SRC, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on {os.path.basename(CALLS_SRC)}:\n{r.stderr[-4000:]}")
    os.replace(tmp, CALLS)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":  # pragma: no cover
    import sys
    build(force="--force" in sys.argv, verbose=True)
