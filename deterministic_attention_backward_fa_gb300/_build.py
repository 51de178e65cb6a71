"""Builds libdash.so in-tree with nvcc for sm_103a.

Each translation unit compiles in its own nvcc process (in parallel); the
objects go to ``_build/`` beside this file and the shared library next to the
package's ``__init__``, with the compiled part of the Python binding (named by
the torch version and the interpreter that it is compiled against).  The library links the CUDA runtime statically and
reaches the driver (for tensor-map encoding) through the runtime's
entry-point query, so it loads on machines without a GPU driver.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdash.so")

SOURCES = ["api.cpp", "schedule.cpp", "place.cpp", "packed_api.cpp", "packed_plan.cpp", "bwd.cu", "fwd.cu",
           "noalloc.cu", "place.cu", "packed_fwd.cu", "packed_bwd.cu", "paged.cu", "ops_api.cpp", "norm_rope.cu",
           "cache8_api.cpp", "cache8.cu", "decode8.cu", "shared.cu"]
BINDING = "binding.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libdash.so")


def binding_path() -> str:
    """The compiled part of the binding for the torch and the interpreter of this process."""
    import torch
    return os.path.join(PKG, f"_binding_{torch.__version__.replace('+', '_')}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_lacks() -> str | None:
    """What this machine lacks for the compiled part of the binding, or None.  The C ABI needs none of it, and the
    Python form of the calls stands in for the compiled one."""
    try:
        import torch
    except ImportError:
        return "torch"
    for path in (os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd", "python_variable.h"),
                 os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(path):
            return path
    return None if shutil.which("g++") else "g++"


def _torch_flags():
    import torch
    top = os.path.dirname(torch.__file__)
    inc = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    abi = int(torch.compiled_with_cxx11_abi())
    return ([x for i in inc for x in ("-I", i)] + [f"-D_GLIBCXX_USE_CXX11_ABI={abi}"],
            ["-L", os.path.join(top, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "dash.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    made = [LIB] if binding_lacks() else [LIB, binding_path()]
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src + ".o")
        cmd = [cc, *ARCH, *COMMON, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cu"):
            cmd.insert(1, "-Xptxas=-v" if verbose else "-Xptxas=-warn-spills")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return obj, (r.stdout + r.stderr)

    lacks = binding_lacks()
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for (_, log) in results:
            if log.strip():
                print(log)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # the library stands by now, whatever becomes of the binding
    if lacks:
        warnings.warn(f"the compiled part of the Python binding is left out: this machine lacks {lacks}")
    else:
        _link_binding(*binding.result())
    return LIB


def _compile_binding():
    """Compiles the binding; its object and the libraries that it links against."""
    flags, libs = _torch_flags()
    obj = os.path.join(BUILD, BINDING + ".o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", *flags, "-c", os.path.join(CSRC, BINDING), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj, libs


def _link_binding(obj, libs):
    tmp = binding_path() + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:" + os.path.basename(LIB), *libs, "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, binding_path())


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
