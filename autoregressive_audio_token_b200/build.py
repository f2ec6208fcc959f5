"""Build libm3.so (the CUDA C-ABI library) in-tree for sm_100a, and _ops (the
native Python binding of its serving operators).

Each .cu translation unit is compiled by its own nvcc process (in parallel),
then linked into autoregressive_audio_token_b200/libm3.so with the CUDA
runtime linked statically.  The binding is one C++ file against torch's
headers, compiled beside them and linked to libm3.so; without those or a C++
compiler the library is built alone.
"""
from __future__ import annotations

import concurrent.futures as cf
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
LIB = os.path.join(PKG, "libm3.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]

SOURCES = ["m3.cu", "attention.cu", "gemv_tile.cu", "gemv_bf16.cu", "gemv_i8row.cu",
           "gemv_i8g128.cu", "gemm_tc.cu", "dit.cu", "dit_gemm.cu", "depth.cu", "ops.cu", "ops_attn.cu"]


BINDING_SRC = os.path.join(CSRC, "ops_binding.cpp")
BINDING = os.path.join(PKG, "_ops" + sysconfig.get_config_var("EXT_SUFFIX"))


def _deps_mtime() -> float:
    files = ([os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")] +
             [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)])
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, extra: list[str], bdir: str = BUILD) -> str:
    obj = os.path.join(bdir, os.path.splitext(src)[0] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _binding_lacks() -> str | None:
    """What the binding needs and this machine does not have (libm3.so needs none of it)."""
    torch = importlib.util.find_spec("torch")
    if torch is None:
        return "torch"
    for header in (os.path.join(torch.submodule_search_locations[0], "include", "torch", "csrc", "utils", "pybind.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return header
    cxx = os.environ.get("CXX", "g++")
    return None if shutil.which(cxx) else cxx


def _compile_binding(force: bool) -> str | None:
    """ops_binding.cpp's object where it is newer than the module, else None; None too where it
    cannot be built here (said on stderr), and then a module older than its sources is removed."""
    deps = [BINDING_SRC, os.path.abspath(__file__)] + \
        [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    if not force and os.path.exists(BINDING) and \
            os.path.getmtime(BINDING) >= max(os.path.getmtime(f) for f in deps):
        return None
    if lacks := _binding_lacks():
        sys.stderr.write(f"_ops, the binding of the serving operators, is not built: {lacks} is missing\n")
        if os.path.exists(BINDING) and os.path.getmtime(BINDING) < max(os.path.getmtime(f) for f in deps):
            os.remove(BINDING)
        return None
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, "ops_binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-DTORCH_EXTENSION_NAME=_ops", "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for ops_binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    torch_lib = os.path.join(importlib.util.find_spec("torch").submodule_search_locations[0], "lib")
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libm3.so",
           "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose_ptxas: bool = False, out: str | None = None,
          defines: tuple = (), build_dir: str | None = None) -> str:
    """Compile libm3.so; `defines` (e.g. ("M3_STAGES=4",)) and `out` build a
    variant elsewhere for tuning sweeps."""
    lib = out or LIB
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _deps_mtime():
        if out is None and (obj := _compile_binding(force)):
            _link_binding(obj)
        return lib
    bdir = build_dir or BUILD
    os.makedirs(bdir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    extra += [f"-D{d}" for d in defines]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, force) if out is None else None
        objs = list(ex.map(lambda s: _compile(s, extra, bdir), SOURCES))
    tmp = lib + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if binding is not None and (obj := binding.result()):
        _link_binding(obj)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas" in sys.argv))
