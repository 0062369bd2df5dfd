"""Builds libsplitkv.so in-tree with nvcc for sm_103a, and beside it the Python
module that marshals the cache operators' torch arguments (no cmake)."""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsplitkv.so")
SOURCES = ["plan.cpp", "api.cu", "gqa_decode.cu", "mla_decode.cu", "combine.cu", "noalloc.cu",
           "refresh.cu", "cache_api.cu", "append.cu", "key_weights.cu", "evict.cu",
           "cross_attend.cu"]
BINDING = os.path.join(PKG, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps() -> list:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "splitkv.h"))
    files.append(os.path.abspath(__file__))
    return files


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(f) > t for f in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compiles every source (in parallel) and links libsplitkv.so (its path is
    returned) and _binding.so."""
    if not force and not is_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
              "--expt-relaxed-constexpr"] + ARCH
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, "-c", os.path.join(CSRC, src), "-o", obj] + common
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_verbose:
            print(r.stdout + r.stderr)
        return obj

    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    binding_obj = os.path.join(BUILD, "binding.o")

    def run(what, cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")

    def compile_binding():
        run("g++ on binding.cpp", ["g++", "-c", os.path.join(CSRC, "binding.cpp"), "-o", binding_obj, "-O2", "-std=c++17",
                                   "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
                                   "-isystem", os.path.join(torch, "include"),
                                   "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include")])

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # (torch's libraries are loaded by then: the package imports torch first)
    tmp = BINDING + ".tmp"
    run("linking _binding.so", ["g++", "-shared", "-o", tmp, binding_obj, "-L", PKG, "-l:libsplitkv.so", "-Wl,-rpath,$ORIGIN",
                                "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
