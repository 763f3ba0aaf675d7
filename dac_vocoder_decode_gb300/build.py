"""In-tree build of the CUDA library libvocoder.so (sm_103a only).

    python -m dac_vocoder_decode_gb300.build            # build if sources changed
    python -m dac_vocoder_decode_gb300.build --force    # rebuild
"""
from __future__ import annotations

import argparse
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
LIB = os.path.join(LIBDIR, "libvocoder.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = LIB + f".tmp{os.getpid()}"
    base = [nvcc(), *(extra or []), *(["-Xptxas=-v"] if verbose else []), *ARCH_FLAGS, "-O3",
            "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE,
            "-I", CSRC]
    # one object per source file, compiled side by side
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [f"{tmp}.{os.path.basename(u)}.o" for u in units]
    try:
        procs = [subprocess.Popen([*base, "-c", "-o", o, u], stdout=subprocess.PIPE,
                                  stderr=subprocess.STDOUT, text=True)
                 for u, o in zip(units, objs)]
        logs = [p.communicate()[0] for p in procs]
        failed = any(p.returncode for p in procs)
        if not failed:
            res = subprocess.run([nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs],
                                 capture_output=True, text=True)
            logs.append(res.stdout + res.stderr)
            failed = res.returncode != 0
        if failed or verbose:
            sys.stderr.write("".join(logs))
        if failed:
            raise RuntimeError("nvcc failed building libvocoder.so")
        os.replace(tmp, LIB)
    finally:
        for f in [*objs, tmp]:
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
