"""Builds libmoeskew.so in-tree with nvcc for sm_100a (no GPU needed to build), and beside it
libmoeskew_args.so, the host code that reads torch tensors (g++, torch's headers; without them
it is left out, and what needs it says so).

    python -m skew_aware_token_b200.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoeskew.so")
ARGS_LIB = os.path.join(PKG, "libmoeskew_args.so")
ARGS_SOURCE = os.path.join(CSRC, "torch_args.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not (_args_left_out() or _args_up_to_date()):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _args_left_out() -> str | None:
    """Why libmoeskew_args.so cannot be built here, or None where it can."""
    if importlib.util.find_spec("torch") is None:
        return "torch is not installed"
    if not os.path.exists(os.path.join(_torch_dir(), "include", "torch", "csrc")):
        return "torch has no headers"
    return None if shutil.which(_cxx()) else f"{_cxx()} is not found"


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError(f"{ARGS_SOURCE} needs torch's headers: torch is not installed")
    return spec.submodule_search_locations[0]


def args_target() -> str:
    """What libmoeskew_args.so reads the objects of: this interpreter's torch and its ABI."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        versions = re.findall(r"^(?:__version__|git_version) = '([^']*)'", f.read(), re.M)
    return " ".join(["torch", *versions, str(sysconfig.get_config_var("SOABI"))])


def args_built_for() -> str | None:
    """args_target() of the build that made libmoeskew_args.so (None: there is no such file, or
    it does not say).  The library itself is not loaded."""
    if not os.path.exists(ARGS_LIB):
        return None
    with open(ARGS_LIB, "rb") as f:
        found = re.search(rb"moeskew_args built for \[([^\]]*)\]", f.read())
    return found.group(1).decode() if found else None


def _args_up_to_date() -> bool:
    return args_built_for() == args_target() and all(
        os.path.getmtime(p) <= os.path.getmtime(ARGS_LIB)
        for p in [ARGS_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h")))


def _build_args() -> None:
    """libmoeskew_args.so: linked to the torch that this interpreter imports."""
    torch_dir = _torch_dir()
    include = os.path.join(torch_dir, "include")
    lib = os.path.join(torch_dir, "lib")
    tmp = ARGS_LIB + ".tmp"
    cmd = [_cxx(), "-O3", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f'-DMOESKEW_BUILT_FOR="{args_target()}"', "-I", INCLUDE, "-I", include, "-I",
           os.path.join(include, "torch", "csrc", "api", "include"), "-I",
           sysconfig.get_paths()["include"], ARGS_SOURCE, "-o", tmp, "-L", lib,
           "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {ARGS_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ARGS_LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles every CUDA source of the library and links libmoeskew.so; returns its path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        left_out = _args_left_out()
        args = None
        if left_out:
            sys.stderr.write(f"{os.path.basename(ARGS_LIB)} is left out: {left_out}\n")
        elif force or not _args_up_to_date():
            args = ex.submit(_build_args)
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if args:
        args.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
