"""Builds libmnb.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel to an object under ``_build/``;
the objects link into ``libmnb.so`` next to this file, with the CUDA runtime
linked statically so the library does not depend on which runtime another
package in the process loaded. Beside it goes ``_mnb_py.<key>.so``, the part of
the Python binding that reads tensors through torch's C++ interface; it calls
``libmnb.so`` (found next to it) and holds no computation. The key stands for the
interpreter and the torch that it was made for. ``libmnb.so`` needs
nvcc alone: it is linked first, and without torch it is all that is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import zlib

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libmnb.so")
PY_SRC = os.path.join(CSRC, "py_attn.cpp")
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


def _gxx() -> str:
    return shutil.which("g++") or "g++"


def _torch_dir() -> str | None:
    """Where torch is installed, without importing it; None: it is not."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _py_key(torch_dir: str) -> str:
    """The interpreter and the torch that the Python binding's native part is
    compiled for and linked to, in the names of its object and module: no other
    process finds them."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        made_for = (sysconfig.get_config_var("SOABI") or "") + torch_dir + f.read()
    return f"{zlib.crc32(made_for.encode()):08x}"


def py_path() -> str:
    """The module of this process's interpreter and torch."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        raise RuntimeError("torch not found: the Python binding is built against it")
    return os.path.join(os.path.dirname(LIB_PATH), f"_mnb_py.{_py_key(torch_dir)}.so")


def _compile_py(torch_dir: str, force: bool) -> str:
    """The object of the Python binding's native part."""
    obj = os.path.join(OBJ_DIR, f"py_attn.{_py_key(torch_dir)}.o")
    if not force and not _stale(obj, [PY_SRC, HEADER]):
        return obj
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = os.path.join(torch_dir, "include")
    tmp = f"{obj}.tmp{os.getpid()}"
    cmd = [_gxx(), "-O2", "-std=c++20", "-fPIC", "-fvisibility=hidden", "-w",
           "-isystem", include, "-isystem", os.path.join(include, "torch/csrc/api/include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           "-c", PY_SRC, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {PY_SRC}:\n{res.stdout}{res.stderr}")
    os.replace(tmp, obj)
    return obj


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libmnb.so. What fails in the
    Python binding's native part is raised once libmnb.so is there."""
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

    torch_dir = _torch_dir()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        py = ex.submit(_compile_py, torch_dir, force) if torch_dir else None
        list(ex.map(compile_one, zip(srcs, objs)))

    if force or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}{res.stderr}")
        os.replace(tmp, LIB_PATH)

    if py is None:
        return LIB_PATH
    py_obj, py_so = py.result(), py_path()
    if force or _stale(py_so, [py_obj]):
        torch_lib = os.path.join(torch_dir, "lib")
        tmp = py_so + f".tmp{os.getpid()}"
        cmd = [_gxx(), "-shared", "-o", tmp, py_obj, "-L" + PKG, "-l:libmnb.so", "-L" + torch_lib,
               "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
               "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}{res.stderr}")
        os.replace(tmp, py_so)
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(verbose=True))
