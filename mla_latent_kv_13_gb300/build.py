"""Build libmla.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc.

Each translation unit under csrc/ is compiled in parallel, then linked into
mla_latent_kv_13_gb300/libmla.so (CUDA runtime linked statically). Beside it the Python module
_binding.so (csrc/binding.cpp, against this machine's Python and PyTorch), linked to libmla.so:
after it, and only where PyTorch is there, so that the C library needs no more than nvcc.
Run: python -m mla_latent_kv_13_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmla.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_TAG = os.path.join(BUILD, "binding.tag")  # what _binding.so is tied to
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _cuda_home() -> str:
    nvcc = _nvcc()
    return os.path.dirname(os.path.dirname(nvcc)) if os.path.isabs(nvcc) else "/usr/local/cuda"


def _deps(*patterns):
    return sorted(p for d in (CSRC, INCLUDE) for e in patterns for p in glob.glob(os.path.join(d, e)))


def _newer(made, deps) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(d) <= os.path.getmtime(made) for d in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _deps("*.cu", "*.cuh", "*.h"))


def _tied_to() -> str | None:
    """The Python and the PyTorch that a binding made now is tied to; None without PyTorch."""
    try:
        import torch
    except ImportError:
        return None
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__}"


def binding_up_to_date() -> bool:
    """Newer than its sources, and made for this Python and this PyTorch."""
    if not _newer(BINDING, _deps("*.cpp", "mla.h")):
        return False
    try:
        with open(BINDING_TAG) as f:
            return f.read() == _tied_to()
    except OSError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and (_tied_to() is None or binding_up_to_date())


def _compile_binding() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(_cuda_home(), "include"),
           "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".{os.getpid()}.tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libmla.so", "-Wl,-rpath,$ORIGIN",
           f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def _build_library(verbose: bool, extra_flags) -> None:
    nvcc = _nvcc()
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(sources))) as ex:
        objs = list(ex.map(compile_one, sources))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    tag = _tied_to()
    library = force or not library_up_to_date()
    binding = tag is not None and (force or not binding_up_to_date())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        if library:
            _build_library(verbose, extra_flags)
        if binding:  # its failure leaves the library standing
            _link_binding(obj.result())
            with open(BINDING_TAG, "w") as f:
                f.write(tag)
    if tag is None:
        print("no PyTorch: libmla.so without the Python module _binding.so", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    flags = ["-Xptxas", "-v"] if v else []
    print(build(force="--force" in sys.argv or v, verbose=v, extra_flags=flags))
