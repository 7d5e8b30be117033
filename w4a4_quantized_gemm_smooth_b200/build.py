"""Build the C-ABI library libsvdq.so in-tree for sm_100a.

    python -m w4a4_quantized_gemm_smooth_b200.build [--force] [--verbose]

Every .cu/.cpp under csrc/ is compiled by nvcc (-gencode
arch=compute_100a,code=sm_100a -lineinfo -O3) and linked into
w4a4_quantized_gemm_smooth_b200/_lib/libsvdq.so.  nvcc cross-compiles; no GPU
is needed.  Objects go to _build/ at the repository root and are rebuilt
only when a source or header is newer.  pyext/fastcall.c becomes
_lib/_svdq_fastcall with the running interpreter's suffix, the CPython binding
of the shortest calls.
"""
from __future__ import annotations

import argparse
import concurrent.futures
import glob
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
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libsvdq.so")
FASTCALL_SRC = os.path.join(PKG, "pyext", "fastcall.c")
# named for the interpreter it is built for: another one builds its own beside it
FASTCALL = os.path.join(LIB_DIR, "_svdq_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
HOST_FLAGS = "-fPIC,-fopenmp,-O3,-ffp-contract=off,-fno-fast-math"
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-I", INCLUDE, "-I", CSRC,
          "-Xcompiler", HOST_FLAGS]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the library needs the CUDA toolkit to build")
    return cand


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    nvcc = _nvcc()
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    headers = (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
               glob.glob(os.path.join(INCLUDE, "*.h")))
    hdr_time = _newest(headers) if headers else 0.0
    objs, jobs = [], []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if (not force and os.path.exists(obj) and
                os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_time)):
            continue
        cmd = [nvcc, *ARCH, *COMMON, "-c", src, "-o", obj]
        if src.endswith(".cu") and verbose:
            cmd += ["-Xptxas", "-v"]
        jobs.append((src, cmd))

    def compile_one(job):
        return job, subprocess.run(job[1], capture_output=True, text=True)

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        for (src, cmd), res in pool.map(compile_one, jobs):
            if verbose:
                print(" ".join(cmd), flush=True)
            if verbose or res.returncode != 0:
                sys.stdout.write(res.stdout)
                sys.stderr.write(res.stderr)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest(objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-Xcompiler", "-fopenmp",
               "-lcudart", "-lgomp"]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stdout.write(res.stdout)
            sys.stderr.write(res.stderr)
            raise RuntimeError("link of libsvdq.so failed")
    build_fastcall(force, verbose)
    return LIB


def build_fastcall(force: bool = False, verbose: bool = False) -> bool:
    """Build the CPython binding of the 16-bit operators.  It wants gcc and the
    interpreter's headers; without them the library and the quantised layers
    work all the same, so a failure is reported and not raised: the first call
    of a 16-bit operator raises, and no module of an older build is left."""
    deps = [FASTCALL_SRC, os.path.join(INCLUDE, "svdq.h")]
    if not force and os.path.exists(FASTCALL) and os.path.getmtime(FASTCALL) >= _newest(deps):
        return True
    cmd = ["gcc", "-O2", "-Wall", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], FASTCALL_SRC, "-o", FASTCALL,
           "-L", LIB_DIR, "-lsvdq", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
        ok, said = res.returncode == 0, res.stdout + res.stderr
    except OSError as e:
        ok, said = False, f"{e}\n"
    if verbose or not ok:
        sys.stderr.write(said)
    if not ok:
        if os.path.exists(FASTCALL):
            os.remove(FASTCALL)
        sys.stderr.write(f"{os.path.basename(FASTCALL)} was not built: the 16-bit operators cannot be "
                         "called from Python (gcc and Python's headers build it)\n")
    return ok


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
