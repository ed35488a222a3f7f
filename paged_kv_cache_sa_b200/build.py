"""Build ``lib/libsa.so`` from ``csrc/*.cu`` with nvcc for sm_100a (in-tree, no JIT cache).

Each translation unit is compiled in parallel, then linked into one shared library
that exports only the C ABI declared in ``include/sa.h``.  The CUDA runtime is linked
statically; the driver's tensor-map encoder is resolved at run time, so the library
has no link-time dependency on libcuda.  ``lib/_binding.*.so`` (csrc/binding.cpp, g++) is the part
of the Python binding that looks into torch tensors; it links torch and Python, not CUDA, and
carries their versions in its name, so that another torch finds no file of the old one.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
OBJDIR = os.path.join(PKG, "lib", "obj")
LIB = os.path.join(LIBDIR, "libsa.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=(), trace: bool = False) -> str:
    """Compile every csrc/*.cu and link lib/libsa.so; returns the library path.  trace:
    the same sources with -DSA_TRACE (phase-timeline points, include/sa_trace.h) into
    lib/libsa_trace.so instead."""
    objdir = OBJDIR + ("_trace" if trace else "")
    lib = os.path.join(LIBDIR, "libsa_trace.so") if trace else LIB
    os.makedirs(objdir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                     + glob.glob(os.path.join(INCLUDE, "*.h")))
    nv = nvcc()
    flags = NVCC_FLAGS + list(extra_flags) + (["-DSA_TRACE"] if trace else [])

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        if force or _stale(obj, [src, __file__] + headers):
            cmd = [nv] + ARCH + flags + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    if force or _stale(lib, objs):
        tmp = lib + ".tmp.%d" % os.getpid()
        cmd = [nv] + ARCH + ["-shared", "-o", tmp] + objs + ["-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
        os.replace(tmp, lib)
    if not trace:
        build_binding(force)
    return lib


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp into lib/_binding.<python>.torch-<version>.so."""
    import sysconfig
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    path = os.path.join(LIBDIR, "_binding.%s.torch-%s.so"
                        % (sys.implementation.cache_tag, torch.__version__))
    if force or _stale(path, [src, __file__, os.path.join(INCLUDE, "sa.h")]):
        t = os.path.dirname(torch.__file__)
        inc = [INCLUDE, os.path.join(t, "include"),
               os.path.join(t, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_path("include")]
        tmp = path + ".tmp.%d" % os.getpid()
        cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi()]
               + [x for d in inc for x in ("-I", d)]
               + [src, "-o", tmp, "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu",
                  "-lc10"])
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("g++ failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        os.replace(tmp, path)
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, trace="--trace" in sys.argv))
