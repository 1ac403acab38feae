"""Builds liblmoe.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc.

Each .cu under csrc/ is compiled to an object in parallel, then the objects
are linked into top_routing_mxfp4_gb300/liblmoe.so (CUDA runtime linked
statically).  Beside it, csrc/bind_torch.cpp becomes _lmoe_torch.so, the
binding of the short calls on torch tensors (g++, torch's headers).  Rebuilds
only what is older than its sources and headers, and the binding also when it
was built for another torch or Python.
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblmoe.so")
BIND_SRC = os.path.join(CSRC, "bind_torch.cpp")
BIND = os.path.join(PKG, "_lmoe_torch.so")
BIND_TAG = os.path.join(BUILD, "lmoe_torch.tag")  # what it was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                     "-Xptxas", "-warn-spills", f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the lmoe CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    deps = sources() + [h for p in (os.path.join(CSRC, "*.cuh"), os.path.join(CSRC, "*.h"), os.path.join(ROOT, "include", "*.h"))
                        for h in glob.glob(p)]
    return max(os.path.getmtime(p) for p in deps) > os.path.getmtime(LIB)


def _torch_dir() -> str:
    """The installed torch, located, not imported."""
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def _bind_tag() -> str:
    """What the binding is bound to: this torch and this Python."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        version = re.search(r"^__version__ = ['\"]([^'\"]+)", f.read(), flags=re.M).group(1)
    return f"torch {version}, {sys.implementation.cache_tag}"


def _bind_stale() -> bool:
    deps = [BIND_SRC, os.path.join(ROOT, "include", "lmoe.h")]
    if not os.path.exists(BIND) or max(os.path.getmtime(p) for p in deps) > os.path.getmtime(BIND):
        return True
    try:
        with open(BIND_TAG) as f:
            return f.read() != _bind_tag()
    except OSError:
        return True


def build_bind() -> str:
    """Build _lmoe_torch.so against the installed torch."""
    torch_dir, tag = _torch_dir(), _bind_tag()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    lib = os.path.join(torch_dir, "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f'-DLMOE_BUILT_FOR="{tag}"',
           *(f"-isystem{i}" for i in inc[:4]), f"-I{inc[4]}", BIND_SRC, "-o", tmp, f"-L{lib}", f"-Wl,-rpath,{lib}",
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind_torch.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    os.makedirs(BUILD, exist_ok=True)
    with open(BIND_TAG, "w") as f:
        f.write(tag)
    return BIND


def build(force: bool = False, verbose: bool = False, extra_flags=(), out: str | None = None) -> str:
    """Build liblmoe.so (or, with `extra_flags` such as -DLMOE_TRACE, a
    variant written to `out`, compiled in its own build folder)."""
    lib = out or LIB
    if out is None and (force or _bind_stale()):
        with cf.ThreadPoolExecutor(max_workers=1) as ex:
            binding = ex.submit(build_bind)  # beside the kernels
            built = _build_lib(lib, force, verbose, extra_flags)
            binding.result()
        return built
    return _build_lib(lib, force, verbose, extra_flags)


def _build_lib(lib: str, force: bool, verbose: bool, extra_flags) -> str:
    if not force and not extra_flags and not _stale():
        return LIB
    nvcc = _nvcc()
    bdir = BUILD if not extra_flags else BUILD + "_" + "_".join(f.strip("-").replace("=", "") for f in extra_flags)
    os.makedirs(bdir, exist_ok=True)
    objs = []

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
