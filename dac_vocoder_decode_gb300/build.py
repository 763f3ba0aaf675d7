"""In-tree build of the CUDA library libvocoder.so (sm_103a only) and of lm_torch.so, the compiled
binding of the 8-bit operators for torch tensors.

    python -m dac_vocoder_decode_gb300.build            # build if sources changed
    python -m dac_vocoder_decode_gb300.build --force    # rebuild
"""
from __future__ import annotations

import argparse
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libvocoder.so")
TORCH_LIB = os.path.join(LIBDIR, "lm_torch.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    built = [LIB] + ([TORCH_LIB] if torch_dir() else [])
    if not all(os.path.exists(b) for b in built):
        return False
    t = min(os.path.getmtime(b) for b in built)
    return all(os.path.getmtime(s) <= t for s in sources())


def torch_dir():
    """The installed torch package's folder (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    where = list(spec.submodule_search_locations or []) if spec else []
    return where[0] if where else None


def torch_command(out: str):
    """The compiler call for lm_torch.so."""
    t = torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
            "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), os.path.join(CSRC, "lm_torch.cpp"), "-o", out,
            "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(t, "lib")]


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
    torch_tmp = TORCH_LIB + f".tmp{os.getpid()}"
    try:
        cmds = [[*base, "-c", "-o", o, u] for u, o in zip(units, objs)]
        if torch_dir():
            cmds.append(torch_command(torch_tmp))
        procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                 for c in cmds]
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
            raise RuntimeError("building libvocoder.so or lm_torch.so failed")
        os.replace(tmp, LIB)
        if torch_dir():
            os.replace(torch_tmp, TORCH_LIB)
    finally:
        for f in [*objs, tmp, torch_tmp]:
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
