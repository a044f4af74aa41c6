"""In-tree build of libpagedkv.so for sm_103a with nvcc (no cmake, no torch), and of
_pkv_torch.so, the Python entry points that take torch tensors (g++, torch's headers;
left out where torch is not installed).

Each translation unit compiles in parallel into ``_build/``; the shared
libraries land next to this file.  A rebuild happens when any source or header
is newer than a library, or when torch or Python are not the ones that the binding
was built for.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
BINDING_SRC = os.path.join(CSRC, "binding", "torch_binding.cpp")
BINDING = os.path.join(PKG, "_pkv_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", f"-I{INCLUDE}"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv")
    return exe


def has_torch() -> bool:
    try:
        return importlib.util.find_spec("torch") is not None
    except ValueError:      # a stand-in in sys.modules
        return False


def binding_abi() -> str:
    """What the binding's C++ and Python ABI depend on."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:     # a torch built in place
        import torch
        version = torch.__version__
    return f"torch {version}, {sys.implementation.cache_tag}"


def built_abi():
    """``binding_abi()`` of the binding that is there; None for an unknown one."""
    try:
        with open(BINDING + ".abi") as f:
            return f.read()
    except OSError:
        return None


def sources():
    cu = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    cpp = sorted(glob.glob(os.path.join(CSRC, "*.cpp")))
    deps = cu + cpp + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [BINDING_SRC]
    return cu, cpp, deps


def stale() -> bool:
    built = [LIB, BINDING] if has_torch() else [LIB]
    if not all(os.path.exists(f) for f in built):
        return True
    if has_torch() and built_abi() != binding_abi():
        return True
    t = min(os.path.getmtime(f) for f in built)
    return any(os.path.getmtime(f) > t for f in sources()[2] + [__file__])


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def binding_commands():
    """Compile and link commands of the torch binding."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "torch_binding.cpp.o")
    cxx = os.environ.get("CXX", "g++")
    compile_ = [cxx, *CXX_FLAGS, "-I" + sysconfig.get_paths()["include"],
                *(f"-isystem{os.path.join(root, 'include', d)}"
                  for d in ("", os.path.join("torch", "csrc", "api", "include"))),
                f"-isystem{os.path.join(cuda, 'include')}",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                "-c", BINDING_SRC, "-o", obj]
    lib = os.path.join(root, "lib")
    # torch's libraries are loaded by then: only their names are needed
    link = [cxx, "-shared", "-o", BINDING + ".tmp", obj, f"-L{PKG}", "-lpagedkv", f"-L{lib}",
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build_library(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every CUDA / C++ unit for sm_103a and link ``libpagedkv.so``, then, where torch is
    installed, the torch binding against it."""
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cu, cpp, _ = sources()
    nv = nvcc()
    jobs = []
    for src in cu:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        extra = ["-Xptxas", "-v"] if verbose_ptxas else []
        jobs.append([nv, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj])
    for src in cpp:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        jobs.append([os.environ.get("CXX", "g++"), *CXX_FLAGS, "-c", src, "-o", obj])
    objs = [j[-1] for j in jobs]
    bind_link = None
    if has_torch():
        bind, bind_link = binding_commands()
        jobs.append(bind)
    logs = []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for out in ex.map(_run, jobs):
            logs.append(out)
    tmp = LIB + ".tmp"
    _run([nv, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    if bind_link:
        _run(bind_link)
        os.replace(BINDING + ".tmp", BINDING)
        with open(BINDING + ".abi", "w") as f:
            f.write(binding_abi())
    if verbose_ptxas:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write("\n".join(logs))
    return LIB


if __name__ == "__main__":
    print(build_library(force=True, verbose_ptxas="-v" in sys.argv))
