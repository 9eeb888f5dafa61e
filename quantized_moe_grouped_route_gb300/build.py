"""Build libqmoe.so (the CUDA kernels and the C-ABI) in-tree for sm_103a, and qmoe_torch.so,
the compiled part of operators.py.

Each .cu file is compiled in parallel with nvcc, then linked into
``quantized_moe_grouped_route_gb300/_lib/libqmoe.so``, which needs nothing of PyTorch; the host
compiler builds ``_lib/qmoe_torch.so`` against it, PyTorch and Python, anew for another
PyTorch or Python (``_build/qmoe_torch.for`` says which it was built for), and not at all where
PyTorch has no CUDA (operators.py then says so when it is used).  Runs on a machine without a
GPU (nvcc cross-compiles).  ``python -m quantized_moe_grouped_route_gb300.build``.
"""

from __future__ import annotations

import concurrent.futures
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
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libqmoe.so")
BINDING = os.path.join(LIBDIR, "qmoe_torch.so")
BINDING_FOR = os.path.join(BUILD, "qmoe_torch.for")

SOURCES = ["api.cu", "route.cu", "misc.cu", "gemm.cu", "gemm2.cu", "api_ops.cu", "gate.cu",
           "tokens.cu", "lora.cu", "lora_shrink.cu", "lora_gemm.cu", "api_block.cu", "norm.cu",
           "norm_backward.cu", "checkpoint.cu", "ffn_gemm.cu", "ffn_stream.cu", "ffn_few.cu",
           "ffn_finish.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "qmoe.h")]
    return max(os.path.getmtime(p) for p in paths)


def _torch_version():
    """What qmoe_torch.so is built for: PyTorch's and Python's versions; None without a
    PyTorch that has CUDA."""
    try:
        import torch
    except ImportError:
        return None
    return f"{torch.__version__} {sys.version}" if torch.version.cuda else None


def _fresh(path: str, newest: float) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= newest


def _binding_fresh(version: str, newest: float) -> bool:
    if not _fresh(BINDING, newest) or not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        return f.read() == version


def _compile_binding() -> str:
    """binding.cpp to an object file; the linking waits for libqmoe.so."""
    import torch
    from torch.utils import cpp_extension
    includes = [INCLUDE, sysconfig.get_paths()["include"], "/usr/local/cuda/include",
                *cpp_extension.include_paths()]
    obj = os.path.join(BUILD, "binding.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f for d in includes for f in ("-isystem" if d != INCLUDE else "-I", d)],
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str, version: str):
    from torch.utils import cpp_extension
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, LIB,
           *[f"-L{d}" for d in cpp_extension.library_paths()], "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(version)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    newest = _inputs_mtime()
    version = _torch_version()
    want_lib = force or not _fresh(LIB, newest)
    want_binding = version is not None and (force or not _binding_fresh(version, newest))
    if not want_lib and not want_binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding) if want_binding else None
        if want_lib:
            _build_lib(ex, verbose, extra_flags)
        if want_binding:
            _link_binding(binding.result(), version)
    return LIB


def _build_lib(ex, verbose, extra_flags):
    cc = nvcc()
    common = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "-I", CSRC, *extra_flags]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return obj

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-Xlinker",
           "-soname=libqmoe.so"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
