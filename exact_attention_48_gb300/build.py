"""Compile libfa.so in-tree for sm_103a with nvcc (no cmake, no torch build helpers).

    python -m exact_attention_48_gb300.build [--force] [-v]

Each .cu file under csrc/ is compiled in parallel to an object file, then
they are linked into ``_build/libfa.so`` with the CUDA runtime linked
statically.  ``-v`` passes ``-Xptxas -v`` (registers, spills, shared memory).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB = os.path.join(BUILD, "libfa.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return exe


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    return _build_into(BUILD, LIB, [], verbose)


# Test builds: the same sources with extra preprocessor definitions, linked
# into their own folder under _build/ (never into libfa.so).  The one used
# by the tests shortens every pipeline wait to FA_WAIT_LIMIT_NS (1 ms) and
# leaves out one load of a kernel: the first V tile of the forward and of each
# run of the drafted-tree attention (bf16 and 8 bits), the first key block of the key weights of
# few query rows and the first query tile of those of many.  So the bounded-wait
# path (FA_ERR_DEVICE_TIMEOUT through fa_device_status) can be exercised
# without any kernel waiting for long.
VARIANTS = {
    "stalltest": ["-DFA_WAIT_LIMIT_NS=1000000ULL", "-DFA_TEST_SKIP_FIRST_V_LOAD"],
}


def build_variant(name: str, force: bool = False) -> str:
    out_dir = os.path.join(BUILD, name)
    lib = os.path.join(out_dir, "libfa.so")
    if not force and os.path.exists(lib) and all(os.path.getmtime(p) <= os.path.getmtime(lib) for p in _deps()):
        return lib
    return _build_into(out_dir, lib, VARIANTS[name], False)


def _build_into(out_dir: str, lib: str, defines, verbose: bool) -> str:
    os.makedirs(out_dir, exist_ok=True)
    exe = nvcc()
    extra = (["-Xptxas", "-v"] if verbose else []) + list(defines)

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [exe, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    objs = []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        for src, obj, r in ex.map(compile_one, _sources()):
            if verbose or r.returncode:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
            objs.append(obj)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [exe, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"linking {lib} failed")
    os.replace(tmp, lib)
    return lib


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
