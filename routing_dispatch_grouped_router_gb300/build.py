"""Builds libmok.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc, and
the Python module _block (block_binding.cpp: torch tensors to its C calls).

    python -m routing_dispatch_grouped_router_gb300.build

Each translation unit compiles in parallel; the libraries are relinked only when
a source or header is newer than they.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libmok.so")
BINDING = os.path.join(LIB_DIR, "_block" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SRC = os.path.join(CSRC, "block_binding.cpp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _cuda_home(nvcc: str) -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _binding_commands(obj: str, out: str, libdir: str):
    """Compile and link commands of the module, with torch's headers and libraries."""
    import torch
    top = os.path.dirname(torch.__file__)
    inc = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api",
                                                      "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(libdir), "include")]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *["-I" + p for p in inc], "-c", BINDING_SRC, "-o", obj]
    link = [cxx, "-shared", obj, "-o", out, "-L" + LIB_DIR, "-l:libmok.so",
            "-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
            "-ltorch", "-lc10_cuda", "-lc10", "-L" + libdir, "-lcudart", "-Wl,-rpath,$ORIGIN",
            "-Wl,-rpath," + os.path.join(top, "lib"), "-Wl,-rpath," + libdir]
    return compile_, link


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every CUDA source and link lib/libmok.so, compile and link the
    binding against it; returns the library's path."""
    if not force and not ptxas_info and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")

    libdir = os.path.join(_cuda_home(nvcc), "lib64")
    bind_obj = os.path.join(BUILD, "block_binding.o")
    compile_binding, link_binding = _binding_commands(bind_obj, BINDING + ".tmp", libdir)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(16, os.cpu_count() or 1))) as ex:
        bind = ex.submit(run, compile_binding, "block_binding.cpp")
        objs = list(ex.map(compile_one, _sources()))
        bind.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", "-rpath," + libdir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    run(link_binding, "linking the binding")
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
