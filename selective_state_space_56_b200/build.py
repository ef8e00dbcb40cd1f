"""Build libmamba_s6.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m selective_state_space_56_b200.build [--force] [--verbose]

Every .cu under csrc/ is compiled separately (in parallel) with
``-gencode arch=compute_100a,code=sm_100a -O3 -lineinfo`` and linked into
``selective_state_space_56_b200/libmamba_s6.so`` with the CUDA runtime linked
statically, so the library loads next to any PyTorch build.  Objects and the
``-Xptxas -v`` report go to ``_build/`` at the repository root.

``csrc/binding.cpp`` (native argument checks and allocations for the layer operators) is
compiled with g++ against the interpreter's own PyTorch into ``_native-<its version>.so`` beside
it, so that another PyTorch gets a binding of its own.  It is optional: where it cannot be built,
``build`` says so and the library is complete without it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libmamba_s6.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
BINDING = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG, "_native-%s.so" % torch.__version__)

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I" + CSRC, "-I" + INCLUDE]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmamba_s6.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                              glob.glob(os.path.join(CSRC, "*.h")) +
                              glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _build_binding(force: bool) -> None:
    header = os.path.join(INCLUDE, "mamba_s6.h")
    if (not force and os.path.exists(BINDING_PATH)
            and os.path.getmtime(BINDING_PATH) >= max(map(os.path.getmtime, (BINDING, header)))):
        return
    from torch.utils import cpp_extension
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], INCLUDE]
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    lib = cpp_extension.library_paths()[0]
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
            '-DS6_TORCH_VERSION="%s"' % torch.__version__] + ["-I" + d for d in inc + [cuda]] +
           [BINDING, "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on %s:\n%s" % (BINDING, r.stderr))
    os.replace(tmp, BINDING_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    path = _build_library(force, verbose)
    try:
        _build_binding(force)
    except Exception as e:  # no g++, no torch headers, a torch without CUDA: the library does without
        if os.path.exists(BINDING_PATH):  # made for other sources
            os.remove(BINDING_PATH)
        warnings.warn("%s was not built, its calls go through the interpreter: %s" % (os.path.basename(BINDING_PATH), e))
    return path


def _build_library(force: bool, verbose: bool) -> str:
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, sources()))
    with open(os.path.join(BUILD_DIR, "ptxas_report.txt"), "w") as f:
        for obj, log in results:
            f.write("== %s\n%s\n" % (os.path.basename(obj), log))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(open(os.path.join(BUILD_DIR, "ptxas_report.txt")).read())
    return LIB_PATH


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
