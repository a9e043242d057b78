"""Build libfusedlin.so in-tree with nvcc for sm_103a.

Each translation unit under csrc/ compiles to an object in parallel; the
objects link into gemm_epilogue_tma_gb300/libfusedlin.so (CUDA runtime linked
statically, the driver reached through the runtime's entry-point query, so
the library loads on a machine without a GPU). binding/fl_torch.cpp, the
extension module that passes torch tensors to the serving operators, compiles
beside them with the host compiler into _torch_binding.so, against the torch
that is installed; without one the library is built alone.

    python -m gemm_epilogue_tma_gb300._build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfusedlin.so")
BINDING_SRC = os.path.join(PKG, "binding", "fl_torch.cpp")
BINDING = os.path.join(PKG, "_torch_binding.so")
STAMP = os.path.join(BUILD, "fl_torch.stamp")  # the torch that BINDING was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libfusedlin")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    if not _stale(obj, [src] + _headers()):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _run(what: str, cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch():
    """The installed torch and Python, as text that changes with them; None without torch. (Not imported for it.)"""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    version = os.path.join(os.path.dirname(spec.origin), "version.py")
    with open(version) as f:
        return f"{spec.origin}\n{f.read()}\nPython {sys.version_info[0]}.{sys.version_info[1]}\n"


def _stamped(torch_text) -> bool:
    if not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == torch_text


def _compile_binding(torch_text: str) -> str:
    obj = os.path.join(BUILD, "fl_torch.o")
    if not _stale(obj, [BINDING_SRC] + _headers()) and _stamped(torch_text):
        return obj
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    _run("the binding's compilation",
         [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", root,
          "-I", os.path.join(root, "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
          "-I", sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj])
    return obj


def _link_binding(obj: str) -> None:
    import torch
    tmp = BINDING + ".tmp"
    _run("the binding's link",
         [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-lfusedlin", "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cuda",
          "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Compile csrc/*.cu and link libfusedlin.so, and the binding if there is a torch; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    torch_text = _torch()
    bound = torch_text is None or (not _stale(BINDING, [BINDING_SRC, LIB] if os.path.exists(LIB) else [BINDING_SRC])
                                   and _stamped(torch_text))
    if not force and not _stale(LIB, srcs + _headers()) and bound:
        return LIB
    jobs = jobs or min(len(srcs) + 1, os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        binding = None if torch_text is None else ex.submit(_compile_binding, torch_text)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
        tmp = LIB + ".tmp"
        _run("link", [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs])
        os.replace(tmp, LIB)
        if binding is not None:
            _link_binding(binding.result())
            with open(STAMP, "w") as f:
                f.write(torch_text)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
