"""Builds the CSA library (libcsa.so) in-tree for sm_103a with nvcc.

Each translation unit compiles in parallel to an object file, then nvcc links
the shared library.  No fast-math: RoPE angles reach ~2.7e5 rad and need the
accurate sincosf.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shlex
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libcsa.so")
CHECKS = os.path.join(OUT_DIR, "csa_checks" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", os.path.join(HERE, "..", "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CSA library needs the CUDA toolkit to build")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    objs = []

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *(extra or []), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_checks()
    return LIB


def build_checks() -> str | None:
    """The binding's argument checks as a CPython extension; None where Python's headers or a C compiler that works are
    missing (the binding then checks in Python, a few microseconds a call slower)."""
    if os.path.exists(CHECKS):
        os.remove(CHECKS)
    include = sysconfig.get_paths()["include"]
    why = "no Python.h"
    if os.path.exists(os.path.join(include, "Python.h")):
        tmp = CHECKS + ".tmp"
        try:
            cmd = [*(shlex.split(os.environ.get("CC") or "") or ["gcc"]), "-O2", "-Wall", "-shared", "-fPIC", "-I",
                   include, os.path.join(CSRC, "checks.c"), "-o", tmp]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode == 0 and os.path.exists(tmp):
                os.replace(tmp, CHECKS)
                return CHECKS
            why = f"{' '.join(cmd)} failed\n{r.stdout}{r.stderr}"
        except (OSError, ValueError) as e:  # no such compiler; a CC that does not parse
            why = str(e)
    print(f"the checks in C are left out: {why}", file=sys.stderr)
    return None


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
