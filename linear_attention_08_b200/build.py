"""Build libkda.so (all CUDA sources, sm_100a) in-tree with nvcc, and, where PyTorch is installed,
_binding.so (the native part of the Python binding) with g++.

Usage: python -m linear_attention_08_b200.build [--force] [--no-binding] [-v]
--no-binding: only libkda.so.  Where there is no PyTorch, run this file instead of the module.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_TORCH = os.path.join(BUILD, "_binding.torch")   # the version of PyTorch it was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "kda.h")]


def _newer(out: str, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _binding_deps():
    return [os.path.join(CSRC, "kda_binding.cpp"), os.path.join(ROOT, "include", "kda.h")]


def _torch_version() -> str | None:
    """The installed PyTorch's version, or None; without importing it."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def _binding_up_to_date() -> bool:
    if not _newer(BINDING, _binding_deps()) or not os.path.exists(BINDING_TORCH):
        return False
    with open(BINDING_TORCH) as f:
        return f.read() == _torch_version()


def up_to_date(binding: bool = True) -> bool:
    return _newer(LIB, _deps()) and (not binding or _torch_version() is None or _binding_up_to_date())


def _build_binding() -> None:
    """_binding.so: the native part of the Python binding, over PyTorch's C++ headers."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    inc = include_paths() + [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(NVCC), "..", "include"),
                             os.path.join(ROOT, "include")]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DKDA_TORCH_VERSION="{torch.__version__}"',
           *(x for p in inc for x in ("-isystem", p)), _binding_deps()[0], "-o", tmp,
           *(f"-L{p}" for p in library_paths()), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           f"-L{PKG}", "-l:libkda.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding failed to compile:\n{res.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_TORCH, "w") as f:
        f.write(str(torch.__version__))


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, binding: bool = True) -> str:
    if force or not _newer(LIB, _deps()):
        os.makedirs(BUILD, exist_ok=True)
        with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
            objs = list(ex.map(lambda s: _compile(s, verbose), _sources()))
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, LIB)
    if binding and _torch_version() is not None and (force or not _binding_up_to_date()):
        _build_binding()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, binding="--no-binding" not in sys.argv))
