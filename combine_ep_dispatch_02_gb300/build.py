"""Build libep.so (the CUDA dispatch / combine library) in-tree with nvcc for sm_103a.

Each .cu file compiles in its own nvcc process (in parallel), then one shared link.  The
library links the shared CUDA runtime so it shares the process's runtime with PyTorch.  The
native half of the Python binding, _ep_binding.so, compiles beside them with g++.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libep.so")
SOURCES = ("ep_api.cu", "ep_route.cu", "ep_scatter.cu", "ep_combine.cu", "ep_noalloc.cu",
           "ep_fp8wire.cu", "ep_grouped.cu", "ep_norm.cu", "ep_sort.cu", "ep_matmul.cu")
BINDING = os.path.join(PKG, "_ep_binding.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "_ep_binding.stamp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libep.so")


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + \
           [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_built_for() -> str:
    """What the binding's binary depends on besides its sources: PyTorch's C++ layout and Python's C API."""
    import torch
    return f"torch {torch.__version__}, cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, {sysconfig.get_config_var('SOABI')}\n"


def _binding_stale() -> bool:
    if _stale(BINDING) or not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != _binding_built_for()


def build_binding() -> None:
    """Compile csrc/ep_binding.cpp against the installed PyTorch; it calls libep.so through addresses it
    is given, so it links nothing of it."""
    import torch
    home = os.path.dirname(torch.__file__)
    tmp = BINDING + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "ep_binding.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on ep_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_built_for())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          defines=(), lib_path: str = LIB, build_dir: str = BUILD_DIR) -> str:
    """Compile libep.so; `defines` (e.g. ["EP_COMBINE_STAGES=4"]) and a separate lib_path /
    build_dir let a caller build tuning variants side by side."""
    product = lib_path == LIB and not defines
    if not force and product and not _stale() and not _binding_stale():
        return LIB
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()
    flags = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
             "-I", CSRC] + [f"-D{d}" for d in defines]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        cmd = [cc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding) if product else None
        objs = list(ex.map(compile_one, SOURCES))
        if binding:
            binding.result()
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [cc, "-shared", *ARCH, "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))
