"""Builds libnorm.so in-tree (``_build/``) with nvcc for sm_103a, and the Python
extension that marshals the calls on attention heads with g++, where PyTorch's
headers are (libnorm.so itself is plain C and needs none).

Each translation unit is compiled in parallel, then linked into one shared
library with the CUDA runtime linked statically.  Rebuilds only what changed.
Run as ``python -m normalization_layernorm_rmsnorm_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libnorm.so")

SOURCES = ["api.cu", "noalloc.cu", "dropout.cu",
           "rownorm_f32.cu", "rownorm_f16.cu", "rownorm_bf16.cu",
           "batchnorm_f32.cu", "batchnorm_f16.cu", "batchnorm_bf16.cu",
           "heads_api.cu", "heads_f32.cu", "heads_f16.cu", "heads_bf16.cu"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [*ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def heads_path() -> str:
    """The compiled marshalling (csrc/heads_binding.cpp) for this PyTorch and Python.  It reads
    PyTorch's objects, so one built for others must not be loaded: the name says which."""
    import sysconfig

    import torch
    return os.path.join(BUILD, f"_heads.{sysconfig.get_config_var('SOABI')}.torch{torch.__version__}"
                               f".abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}.so")


def _binding_includes() -> list[str] | None:
    """Directories of the binding's headers; None where g++, PyTorch's headers and CUDA
    library or Python's headers are missing: then there is no binding to build."""
    import sysconfig
    try:
        import torch
    except (ImportError, OSError):  # (its libraries may be missing)
        return None
    home = os.path.dirname(torch.__file__)
    if not os.path.exists(os.path.join(home, "lib", "libc10_cuda.so")):
        return None
    inc = os.path.join(home, "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"]]
    for header in ("torch/csrc/autograd/python_variable.h", "c10/cuda/CUDAStream.h", "Python.h"):
        if not any(os.path.exists(os.path.join(d, header)) for d in dirs):
            return None
    return dirs if shutil.which("g++") else None


def _compile_binding(includes: list[str]) -> str:
    import torch
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "heads_binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           *(x for d in [*includes, cuda] for x in ("-isystem", d)),
           "-c", os.path.join(CSRC, "heads_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for heads_binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    path = heads_path()
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-lnorm", "-L", libs, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every source, link libnorm.so and the binding; returns libnorm.so's path."""
    os.makedirs(BUILD, exist_ok=True)
    dep = _deps_mtime()

    def stale(f):
        return force or not os.path.exists(f) or os.path.getmtime(f) < dep

    includes = _binding_includes()
    lib, heads = verbose_ptxas or stale(LIB), includes is not None and stale(heads_path())
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as pool:
        binding = pool.submit(_compile_binding, includes) if heads else None
        objs = list(pool.map(lambda s: _compile(s, extra), SOURCES)) if lib else []
    if lib:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding:
        _link_binding(binding.result())
    return LIB


def source_digest(files=None) -> str:
    """sha256 of CUDA sources and the public header (names the kernel version
    an ncu capture was taken on): all of them, or the named files of csrc/
    (and "libnorm.h") that one kernel family is built from."""
    import hashlib
    h = hashlib.sha256()
    if files is None:
        files = sorted(glob.glob(os.path.join(CSRC, "*"))) + [os.path.join(INCLUDE, "libnorm.h")]
    else:
        files = [os.path.join(INCLUDE if f == "libnorm.h" else CSRC, f) for f in sorted(files)]
    for f in files:
        h.update(os.path.basename(f).encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas-v" in sys.argv))
