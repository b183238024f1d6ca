"""Build libmka.so (sm_100a) in-tree with nvcc, and the Python binding of its bounded-memory operators.

    python route_kv_memory_b200/_build.py          # incremental
    python route_kv_memory_b200/_build.py --force  # rebuild everything

Run it as a script (or load it by path): importing the package needs the built library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmka.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_TORCH = os.path.join(BUILD, "binding_torch.txt")  # the torch version that BINDING was built against
SOURCES = ["api.cu", "gemm.cu", "memory.cu", "attention.cu", "decode.cu", "noalloc.cu", "api_bounded.cu", "kv8.cu", "tc_gemm.cu", "tc_attention.cu", "block_sparse.cu", "tc_attention_bwd.cu", "backward.cu", "selftest.cu"]
HEADERS = ["common.cuh", "kernels.h", "sm100.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I" + os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the FastMKA CUDA library cannot be built")


def _newest_dep() -> float:
    deps = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "mka.h")]
    return max(os.path.getmtime(p) for p in deps if os.path.exists(p))


def _compile(src: str, force: bool, verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    path = os.path.join(CSRC, src)
    if (not force and os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(path)
            and os.path.getmtime(obj) >= _newest_dep()):
        return obj
    cmd = [nvcc(), *NVCC_FLAGS, "-c", path, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        print(r.stderr, file=sys.stderr)
    return obj


def build_library(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, force, verbose), SOURCES))
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_binding(force)
    return LIB


def binding_is_current(torch_version: str) -> bool:
    """Whether BINDING is newer than its sources and was built against this torch."""
    newest = max(os.path.getmtime(p) for p in (os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "mka.h")))
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < newest or not os.path.exists(BINDING_TORCH):
        return False
    with open(BINDING_TORCH) as f:
        return f.read() == torch_version


def _build_binding(force: bool) -> None:
    """_binding.so: argument marshalling against torch's headers, linked to libmka.so beside it."""
    import importlib.metadata
    version = importlib.metadata.version("torch")  # (without importing it: an up-to-date build takes no time)
    if not force and binding_is_current(version):
        return
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DMKA_TORCH_VERSION="{torch.__version__}"', *("-isystem" + p for p in inc), src, "-o", tmp,
           "-L" + PKG, "-l:libmka.so", "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_TORCH, "w") as f:
        f.write(version)


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
