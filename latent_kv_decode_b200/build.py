"""Build libmla.so in-tree with nvcc for sm_100a, and the binding module _step beside it.

    python -m latent_kv_decode_b200.build            # incremental
    python -m latent_kv_decode_b200.build --force    # rebuild everything

Each ``csrc/*.cu`` compiles to ``_build/*.o`` (only when the source or a
header is newer), then everything links into ``latent_kv_decode_b200/libmla.so``.
``csrc/step_binding.cpp`` (torch's C++ headers, the host compiler) becomes
``latent_kv_decode_b200/_step.so``, linked against that library.
Needs no GPU: nvcc cross-compiles for the B200.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmla.so")
STEP_SRC = os.path.join(CSRC, "step_binding.cpp")
STEP = os.path.join(PKG, "_step.so")
STEP_STAMP = os.path.join(BUILD, "step.built_for")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
           "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def _compile(src: str, force: bool, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if force or not os.path.exists(obj) or os.path.getmtime(obj) < newest:
        cmd = [nvcc()] + ARCH + NVFLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, force, verbose), srcs))
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    build_step(force, verbose)
    return LIB


def built_for() -> str:
    """What _step.so is compiled against, beside its source: torch's C++ classes and Python's C API."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def build_step(force: bool = False, verbose: bool = False) -> str:
    """The C++ binding of the serving-step calls (needs libmla.so).

    Built anew when its source or mla.h is newer, or when it was built for another
    torch or Python; the module carries what it was built for as ``built_for``.
    """
    header = os.path.join(ROOT, "include", "mla.h")
    newest = max(os.path.getmtime(STEP_SRC), os.path.getmtime(header))
    here = built_for()
    last = open(STEP_STAMP).read() if os.path.exists(STEP_STAMP) else None
    if not force and last == here and os.path.exists(STEP) and os.path.getmtime(STEP) >= newest:
        return STEP
    import torch
    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = STEP + ".tmp"
    cmd = ([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DSTEP_BUILT_FOR="{here}"'] + [x for d in inc for x in ("-isystem", d)] +
           [STEP_SRC, "-o", tmp, "-L" + PKG, "-l:" + os.path.basename(LIB), "-L" + os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + os.path.join(tdir, "lib")])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {STEP_SRC}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, STEP)
    os.makedirs(BUILD, exist_ok=True)
    with open(STEP_STAMP, "w") as f:
        f.write(here)
    return STEP


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true", help="print ptxas register/smem usage")
    a = ap.parse_args()
    print(build(a.force, a.verbose))
