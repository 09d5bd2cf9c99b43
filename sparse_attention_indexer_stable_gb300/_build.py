"""Builds the CUDA library in-tree: csrc/*.cu -> _build/libdcp_topk.so (sm_103a),
and the torch side of the 4-bit cache: csrc/kv4_binding.cpp -> _build/_kv4_binding-*.so.

Plain nvcc, one translation unit per subject compiled side by side, no CMake; host code has no
architecture-specific flags so the same source builds on x86_64 and aarch64.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libdcp_topk.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files


# The race-check build: the same library compiled with -DDCP_DEBUG_POISON
# (odd warps delayed after every barrier, shared state overwritten with
# garbage before every reset, indices from shared state clamped; the 4-bit
# cache's waits for copies short, and a copy that it can be told to leave out),
# for the barrier and time-out tests only; it exports the same C ABI.
POISON_LIB_PATH = os.path.join(OUT_DIR, "libdcp_topk_racecheck.so")
POISON_FLAGS = ("-DDCP_DEBUG_POISON",)


def is_stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, extra_flags=(), path: str = LIB_PATH) -> str:
    """Compile the library if missing or older than its sources; returns its path."""
    if not force and not is_stale(path):
        return path
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = path + f".{os.getpid()}.tmp"
    cmd = [_nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--shared",
           "--threads", "0",
           "-Xcompiler", "-fPIC", "-I", INCLUDE, "-o", tmp, *sources(), *extra_flags]
    subprocess.check_call(cmd)
    os.replace(tmp, path)
    return path


def build_race_check(force: bool = False) -> str:
    """The race-check build (see POISON_LIB_PATH); returns its path."""
    return build(force, POISON_FLAGS, POISON_LIB_PATH)


# The torch side of the 4-bit cache's functions: host C++ against torch's and
# Python's headers, so built anew for another torch, its CUDA, or another Python.
def binding_path() -> str:
    import torch

    return os.path.join(OUT_DIR, f"_kv4_binding-{torch.__version__}-cuda{torch.version.cuda}"
                                 f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_binding(force: bool = False) -> str:
    """Compile csrc/kv4_binding.cpp if missing or older than its sources;
    returns its path."""
    path, source = binding_path(), os.path.join(CSRC, "kv4_binding.cpp")
    headers = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    if not force and os.path.exists(path) and all(
            os.path.getmtime(f) <= os.path.getmtime(path) for f in [source, *headers]):
        return path
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        raise RuntimeError("no C++ compiler: set CXX or put g++ on PATH")
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda_dir = os.path.dirname(os.path.dirname(_nvcc()))
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = path + f".{os.getpid()}.tmp"
    subprocess.check_call([
        cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE,
        "-I", os.path.join(torch_dir, "include"),
        "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
        "-I", os.path.join(cuda_dir, "include"), "-I", sysconfig.get_paths()["include"],
        "-o", tmp, source, "-L", os.path.join(torch_dir, "lib"),
        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, path)
    return path
