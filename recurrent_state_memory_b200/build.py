"""Build libgdr.so (the CUDA library) in-tree for sm_100a with nvcc, and _binding.so (the host side of
some of its Python calls) with g++.  The library needs nvcc alone; the binding needs g++ and the
headers of the installed torch, and without those it is left out with a warning.

    python -m recurrent_state_memory_b200.build [--force]
"""
import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdr.so")
LIB_DEBUG = os.path.join(PKG, "libgdr_debug.so")    # with the kernels' index checks
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

BINDING = os.path.join(PKG, "_binding.so")
CXX = os.environ.get("CXX", "g++")

SOURCES = ["gdr.cu", "scan.cu", "norm.cu", "beam.cu"]
OBJ = os.path.join(PKG, "_build")                   # object files, one folder per build kind
BINDING_MADE_FOR = os.path.join(OBJ, "binding.txt") # the torch and Python that _binding.so was built against


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    files.append(os.path.join(INCLUDE, "gdr.h"))
    files.append(os.path.abspath(__file__))
    return files


def _fresh(out, dep):
    """Whether the object file is newer than this file and every source it was made from."""
    if not (os.path.exists(out) and os.path.exists(dep)):
        return False
    files = open(dep).read().replace("\\\n", " ").split(":", 1)[1].split()
    made = os.path.getmtime(out)
    return all(os.path.exists(f) and os.path.getmtime(f) <= made for f in files + [os.path.abspath(__file__)])


def _torch_and_python() -> str:
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def build_binding(force: bool = False) -> str:
    """Build _binding.so (csrc/binding.cpp) against the installed torch; built again when that changes."""
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    made_from = [src, os.path.join(INCLUDE, "gdr.h"), os.path.abspath(__file__)]
    made_for = _torch_and_python()
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(map(os.path.getmtime, made_from)) \
            and os.path.exists(BINDING_MADE_FOR) and open(BINDING_MADE_FOR).read() == made_for:
        return BINDING
    from torch.utils import cpp_extension
    paths = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(
        os.path.dirname(NVCC)), "include")]
    for header in ("torch/extension.h", "Python.h"):
        if not any(os.path.exists(os.path.join(p, header)) for p in paths):
            raise FileNotFoundError(f"{header} is not installed")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE]
    for p in paths:
        cmd += ["-isystem", p]
    cmd += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DGDR_BUILT_WITH_TORCH="{torch.__version__}"', src, "-o", tmp, "-L", libs,
            "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10", "-lc10_cuda", "-ldl"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    os.makedirs(OBJ, exist_ok=True)
    with open(BINDING_MADE_FOR, "w") as f:
        f.write(made_for)
    return BINDING


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Build libgdr.so (and _binding.so), or with debug=True libgdr_debug.so (-DGDR_BOUNDS_CHECK: the kernels
    test the indices at their GDR_INB marks, which stand at global-memory accesses whose index is
    computed, and report a failure through the status word instead of making the access; what a tensor
    map or a loop's own bound keeps inside has no mark)."""
    if debug:
        return _build_library(LIB_DEBUG, force, verbose, True)
    lib = _build_library(LIB, force, verbose, False)
    try:
        build_binding(force)
    except (ImportError, FileNotFoundError) as e:       # no torch, no headers, no compiler
        warnings.warn(f"_binding.so is not built, gdr's calls of the scan, layer norm and beam search will not work: {e}")
    return lib


def _build_library(lib, force, verbose, debug) -> str:
    if not force and os.path.exists(lib):
        newest = max(os.path.getmtime(f) for f in _deps())
        if os.path.getmtime(lib) >= newest:
            return lib
    obj = os.path.join(OBJ, "debug" if debug else "default")
    os.makedirs(obj, exist_ok=True)
    common = [NVCC, "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
    if debug:
        common.append("-DGDR_BOUNDS_CHECK")
    if verbose:
        common.append("-Xptxas=-v")

    def compile_one(src):
        out = os.path.join(obj, src + ".o")
        dep = out + ".d"
        if not force and _fresh(out, dep):
            return out
        subprocess.run(common + ["-MD", "-MF", dep, "-c", "-o", out, os.path.join(CSRC, src)], check=True)
        return out

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:     # nvcc processes, side by side
        objects = list(pool.map(compile_one, SOURCES))
    tmp = lib + ".tmp"
    subprocess.run(common[:6] + ["-shared", "-o", tmp] + objects, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
