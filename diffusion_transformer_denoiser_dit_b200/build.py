"""Build the in-tree CUDA library libdit_b200.so for sm_100a with nvcc.

Usage: python -m diffusion_transformer_denoiser_dit_b200.build
Objects go to _build/ at the repository root; the shared library is written next
to this file so it travels with the package, and so is _fastcall.so, the short way of binding.py
into it, where Python's and torch's headers are at hand (binding.py does without it otherwise).
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdit_b200.so")
FASTCALL = os.path.join(PKG, "_fastcall.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _needs(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "dit.h"))
    jobs = []
    for src in sources():
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        if _needs(obj, [src] + headers):
            cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", src, "-o", obj]
            jobs.append(cmd)
    objs = [os.path.join(OBJDIR, os.path.basename(s)[:-3] + ".o") for s in sources()]

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or ptxas_verbose or r.returncode != 0:
            sys.stdout.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("compiler failed: " + " ".join(cmd))

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        list(ex.map(run, jobs))
    if jobs or _needs(LIB, objs):
        run([nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", LIB] + objs + ["-lcudart_static", "-ldl", "-lrt", "-lpthread"])
    build_fastcall(verbose or ptxas_verbose)
    return LIB


def build_fastcall(verbose: bool = False):
    """Optional: what cannot be built here is left out with a warning, and an older one does not stay."""
    spec, python = importlib.util.find_spec("torch"), sysconfig.get_paths()["include"]
    src = os.path.join(CSRC, "fastcall.cpp")
    deps = [src, os.path.join(INCLUDE, "dit.h")]
    torch = os.path.dirname(spec.origin) if spec is not None else None
    if torch:
        deps.append(os.path.join(torch, "version.py"))
    if not _needs(FASTCALL, deps):
        return
    if os.path.exists(FASTCALL):
        os.remove(FASTCALL)
    if torch is None or shutil.which("g++") is None or not os.path.exists(os.path.join(python, "Python.h")):
        return
    inc, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE, "-I", python, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, src, "-o", FASTCALL, "-L", lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose:
        sys.stdout.write(r.stdout + r.stderr)
    if r.returncode != 0:
        if os.path.exists(FASTCALL):
            os.remove(FASTCALL)
        sys.stderr.write(r.stderr + "warning: _fastcall.so was not built (calls go through ctypes): " + " ".join(cmd) + "\n")


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, ptxas_verbose="--ptxas" in sys.argv))
