"""Compile libattn.so (the CUDA kernels and the C ABI) in-tree for sm_103a, and _binding.so.

Each .cu file is compiled to an object in parallel with nvcc, then linked into
exact_io_aware_13_gb300/libattn.so. No CMake, no torch extension machinery: the
library exports plain C symbols (include/attn.h). _binding.so is the Python module of the
paged-cache calls (csrc/binding.cpp, compiled against torch's headers by g++); it links to
the library next to it. It holds torch's C++ interface of one version: the version it was
built against is kept beside it, and another one rebuilds it.
"""
from __future__ import annotations

import concurrent.futures
import importlib.metadata
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libattn.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "binding.stamp")

SOURCES = ["attn_api.cu", "simt.cu", "fwd_tc.cu", "fwd256_tc.cu", "bwd_tc.cu", "bwd256_tc.cu", "fp8.cu", "decode_tc.cu",
           "decode_copies2.cu", "paged_cache.cu", "paged_attn.cu", "paged_rows.cu",
           "paged_tiles_bf16.cu", "paged_tiles_e4m3.cu", "pool.cu", "pool_copy.cu", "verify.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (CUDA toolkit required to build libattn.so)")
    return cand


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths.append(os.path.join(INCLUDE, "attn.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _binding_target() -> str:
    """What _binding.so is built for: torch's and Python's versions."""
    return f"torch {importlib.metadata.version('torch')} {sys.implementation.cache_tag}"


def _binding_is_for_this_torch() -> bool:
    try:
        with open(BINDING_STAMP) as f:
            return f.read() == _binding_target()
    except OSError:
        return False


def _compile(src: str, extra: list[str], verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, file=sys.stderr)
    return obj


def _compile_binding(verbose: bool) -> str:
    """binding.cpp to an object; torch tells where its headers are."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    obj = os.path.join(BUILD_DIR, "binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wno-attributes",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-c", os.path.join(CSRC, "binding.cpp"),
           "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "lib64")
    tmp = BINDING_PATH + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libattn.so", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-L", cuda, "-lcudart",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _binding.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_target())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Build libattn.so and _binding.so if a source is newer, _binding.so also if torch is
    another one; return the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= _deps_mtime()
                         for p in (LIB_PATH, BINDING_PATH)):
        if not _binding_is_for_this_torch():
            _link_binding(_compile_binding(verbose))
        return LIB_PATH
    extra = list(extra or [])
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, extra, verbose), SOURCES))
        binding_obj = binding.result()
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_binding(binding_obj)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
