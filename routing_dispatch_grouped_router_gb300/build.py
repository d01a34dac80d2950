"""Builds libmok.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc, and,
where torch is installed, the Python module _block (block_binding.cpp: torch
tensors to its C calls).

    python -m routing_dispatch_grouped_router_gb300.build

Each translation unit compiles in parallel; each of the two is made anew only
when a source or header is newer than it, the module also for another torch.
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


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _library_deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + _headers()


def _newer(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target)
                                          for p in deps)


def _torch():
    """torch with CUDA, or None: the library is built and used without it."""
    try:
        import torch
    except ImportError:
        return None
    return torch if torch.version.cuda else None


def _stamp() -> str:
    """Holds the torch version that the module was compiled against."""
    return BINDING + ".torch"


def _binding_up_to_date(torch) -> bool:
    if torch is None:
        return True
    if not _newer(BINDING, [BINDING_SRC] + _headers()) or not os.path.exists(_stamp()):
        return False
    with open(_stamp()) as f:
        return f.read() == str(torch.__version__)


def up_to_date() -> bool:
    return _newer(LIB, _library_deps()) and _binding_up_to_date(_torch())


def _binding_commands(torch, obj: str, out: str, libdir: str):
    """Compile and link commands of the module, with torch's headers and libraries."""
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
    """Compile every CUDA source and link lib/libmok.so; with torch, compile the
    module and link it against the library.  Returns the library's path."""
    torch = _torch()
    force = force or ptxas_info
    library = force or not _newer(LIB, _library_deps())
    binding = torch is not None and (force or not _binding_up_to_date(torch))
    if not library and not binding:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    libdir = os.path.join(_cuda_home(nvcc), "lib64")

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
        return r

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        r = run([nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj], f"nvcc for {src}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    if binding:
        bind_obj = os.path.join(BUILD, "block_binding.o")
        compile_binding, link_binding = _binding_commands(torch, bind_obj, BINDING + ".tmp", libdir)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(16, os.cpu_count() or 1))) as ex:
        bound = ex.submit(run, compile_binding, "block_binding.cpp") if binding else None
        if library:
            objs = list(ex.map(compile_one, _sources()))
            run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", LIB + ".tmp", *objs,
                 "-Xlinker", "-rpath," + libdir], "link")
            os.replace(LIB + ".tmp", LIB)
        if bound:
            bound.result()
    if binding:
        run(link_binding, "linking the binding")
        os.replace(BINDING + ".tmp", BINDING)
        with open(_stamp(), "w") as f:
            f.write(str(torch.__version__))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
