"""Builds libbinattn.so (the C-ABI library, for sm_100a with nvcc) and _paged (a Python module) in-tree."""
from __future__ import annotations

import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbinattn.so")
MODULE = os.path.join(PKG, "_paged" + sysconfig.get_config_var("EXT_SUFFIX"))  # of this Python
STAMP = os.path.join(BUILD, "paged_built_for")
MODULE_SRC = os.path.join(CSRC, "paged_binding.cpp")
NVCC = os.environ.get("NVCC", "nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(INCLUDE, "binattn.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def installed_torch() -> str:
    """What the Python module is compiled against: it takes tensors apart as this torch lays them out. (Found without
    importing it.)"""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "unknown"


def module_up_to_date() -> bool:
    try:
        with open(STAMP) as f:
            same = f.read() == installed_torch()
    except OSError:
        return False
    deps = [MODULE_SRC, os.path.join(INCLUDE, "binattn.h")]
    return same and os.path.exists(MODULE) and all(os.path.getmtime(f) <= os.path.getmtime(MODULE) for f in deps)


def build_module(force: bool = False) -> str | None:
    """The Python module of the paged cache's entry points, for this interpreter and its torch; None where there is
    no torch (the C library needs none)."""
    if not force and module_up_to_date():
        return MODULE
    try:
        import torch
    except ImportError as e:
        print(f"no Python module of the paged cache's calls: {e}", file=sys.stderr)
        return None
    os.makedirs(BUILD, exist_ok=True)
    home = os.path.dirname(os.path.abspath(torch.__file__))
    tmp = MODULE + f".tmp{os.getpid()}"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(home, "include"), "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBA_BUILT_FOR="torch {torch.__version__}"',
           MODULE_SRC, "-o", tmp, "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {MODULE_SRC}:\n{r.stderr}")
    os.replace(tmp, MODULE)
    with open(STAMP, "w") as f:
        f.write(installed_torch())
    return MODULE


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """The library, and then the Python module where torch is there."""
    path = build_library(force, verbose, ptxas_info)
    build_module(force)
    return path


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose or ptxas_info:
            print(r.stderr, end="")
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_variant(tag: str, defines, force: bool = False) -> str:
    """A test build of the library with extra preprocessor definitions, as
    lib<tag>.so beside the product library (never loaded by the package itself)."""
    out = os.path.join(PKG, f"libbinattn_{tag}.so")
    deps = _deps() + [os.path.abspath(__file__)]
    if not force and os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in deps):
        return out
    bdir = os.path.join(BUILD, tag)
    os.makedirs(bdir, exist_ok=True)
    dflags = [f"-D{d}" for d in defines]

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        r = subprocess.run([NVCC, *ARCH, *FLAGS, *dflags, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
