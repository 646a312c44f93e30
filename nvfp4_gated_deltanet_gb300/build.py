"""Build libgdn.so in-tree for sm_103a: every .cu under csrc/ is compiled in
parallel by nvcc, then linked into one shared library next to this file; and
_kv4.so, the native Python binding of the kv4_* calls, from csrc/kv4_py.cpp."""
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BINDING = os.path.join(PKG, "_kv4.so")
BINDING_SRC = os.path.join(CSRC, "kv4_py.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fno-strict-aliasing",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _binding_object(deps) -> str:
    """Compile the native binding (against the installed PyTorch's headers)."""
    obj = os.path.join(BUILD, "kv4_py.o")
    if not _newer(obj, [BINDING_SRC] + deps):
        torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
        inc = os.path.join(torch_dir, "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-isystem", inc, "-isystem",
              os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem",
              sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj], "g++ on " + BINDING_SRC)
    return obj


def _link_binding(obj: str):
    if not _newer(BINDING, [obj, LIB]):
        tlib = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
        tmp = BINDING + ".tmp"
        _run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libgdn.so", "-Wl,-rpath,$ORIGIN", "-L", tlib,
              "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda"], "linking _kv4.so")
        os.replace(tmp, BINDING)


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if _newer(obj, [src] + headers) and not ptxas_info:
            return obj
        cmd = [cc] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_binding_object, [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)])
        objs = list(ex.map(compile_one, sources()))
        binding = binding.result()
    if not _newer(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _link_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
