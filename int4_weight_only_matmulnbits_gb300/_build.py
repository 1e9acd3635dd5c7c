"""Builds libmnb.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel to an object under ``_build/``;
the objects link into ``libmnb.so`` next to this file, with the CUDA runtime
linked statically so the library does not depend on which runtime another
package in the process loaded. Beside it goes ``_mnb_py.so``, the part of the
Python binding that is written against the CPython C API; it calls
``libmnb.so`` (found next to it) and holds no computation.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libmnb.so")
PY_SRC = os.path.join(CSRC, "py_attn.cpp")
PY_PATH = os.path.join(PKG, "_mnb_py.so")
HEADER = os.path.join(ROOT, "include", "mnb.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmnb.so")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)
            if f.endswith((".cuh", ".h"))] + [HEADER]


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libmnb.so."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = _deps()
    srcs = sources()
    objs = [os.path.join(OBJ_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src_obj):
        src, obj = src_obj
        if not force and not _stale(obj, [src] + headers):
            return obj
        tmp = f"{obj}.tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", tmp]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}{res.stderr}")
        if verbose and res.stderr:
            print(res.stderr)
        os.replace(tmp, obj)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        list(ex.map(compile_one, zip(srcs, objs)))

    if force or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}{res.stderr}")
        os.replace(tmp, LIB_PATH)

    # Python.h's version is part of what the module is built for: another
    # interpreter's is stale.
    stamp = os.path.join(OBJ_DIR, "_mnb_py.abi")
    abi = sysconfig.get_config_var("SOABI") or ""
    old = open(stamp).read() if os.path.exists(stamp) else None
    if force or old != abi or _stale(PY_PATH, [PY_SRC, HEADER]):
        tmp = PY_PATH + f".tmp{os.getpid()}"
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
               "-fvisibility=hidden", "-I" + sysconfig.get_paths()["include"], PY_SRC, "-o", tmp,
               "-L" + PKG, "-l:libmnb.so", "-Wl,-rpath,$ORIGIN"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"g++ failed for {PY_SRC}:\n{res.stdout}{res.stderr}")
        os.replace(tmp, PY_PATH)
        with open(stamp, "w") as f:
            f.write(abi)
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(verbose=True))
