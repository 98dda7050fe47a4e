"""Build libfa.so in-tree with nvcc for sm_103a, and the binding's native part with g++.

Each .cu translation unit is compiled in parallel to an object file, then
the objects are linked into ``libfa.so`` next to this file (the CUDA runtime
is linked statically, the driver API is reached through the runtime's
entry-point query, so the library loads on machines without a GPU).
``_fa_binding.so`` (csrc/fa_binding.cpp) checks and marshals the Python calls of the operators around
cached attention; it is compiled against the installed torch and links ``libfa.so`` beside it.  The
library itself needs neither torch nor g++: ``python exact_tiled_attention_fa_gb300/build.py`` leaves it
there for C callers also where the binding cannot be built.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfa.so")
BINDING = os.path.join(HERE, "_fa_binding.so")
BINDING_SRC = "fa_binding.cpp"
STAMP = os.path.join(BUILD, "fa_binding.host")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _fresh(target, binding):
    """Whether a target is at least as new as its sources: the binding's file, or all others."""
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if (f == BINDING_SRC) == binding] + [os.path.join(INCLUDE, "fa.h")]
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(f) for f in files)


def _host():
    """What the binding was compiled for: it uses torch's and Python's internal C++ interfaces."""
    try:
        import torch
    except ImportError:
        return None  # it cannot be built: the attempt says so
    return f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python {sys.version} {sysconfig.get_platform()}"


def _made_for_host():
    try:
        with open(STAMP) as f:
            return f.read() == _host()
    except OSError:
        return False


def build(force=False, verbose=False, extra_flags=()):
    """Compile every kernel and the C ABI into ``libfa.so``, and the binding; returns the library's path.

    The library needs nvcc alone: it is linked whether or not the binding, which needs torch and a C++
    compiler, can be built.  That raises afterwards.
    """
    library = force or not _fresh(LIB, False)
    binding = force or not _fresh(BINDING, True) or not _made_for_host()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    def link(target, *cmd):
        tmp = target + f".tmp{os.getpid()}"
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, target)

    def compile_binding():
        import torch
        torch_dir = os.path.dirname(torch.__file__)
        obj = os.path.join(BUILD, "fa_binding.o")
        inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
        cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               *[f for i in inc for f in ("-I", i)], "-c", os.path.join(CSRC, BINDING_SRC), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cxx} failed on {BINDING_SRC}:\n{r.stderr}")
        return obj, os.path.join(torch_dir, "lib")

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        made = ex.submit(compile_binding) if binding else None
        if library:
            link(LIB, nvcc, *ARCH, "-shared", "-cudart", "static", *ex.map(compile_one, srcs))
    if made is not None:
        try:
            obj, libs = made.result()
            link(BINDING, cxx, "-shared", obj, "-L", HERE, "-l:libfa.so", "-Wl,-rpath,$ORIGIN", "-L", libs,
                 "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python")
            with open(STAMP, "w") as f:
                f.write(_host())
        except (RuntimeError, ImportError, OSError) as e:
            raise RuntimeError(f"libfa.so is built, _fa_binding.so is not: {e}") from e
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
