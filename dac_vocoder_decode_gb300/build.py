"""In-tree build of the CUDA library libvocoder.so (sm_103a only) and of lm_torch, the compiled
binding of the 8-bit operators for torch tensors.  The library does not need the binding: where that
cannot be built (no C++ compiler, a torch without CUDA), the build says so and goes on, and the
operators are marshalled in Python.

    python -m dac_vocoder_decode_gb300.build            # build if sources changed
    python -m dac_vocoder_decode_gb300.build --force    # rebuild
"""
from __future__ import annotations

import argparse
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

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
    """What libvocoder.so is made of."""
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def torch_sources():
    """What the compiled binding is made of."""
    return sorted(glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def newer(built: str, made_of) -> bool:
    """Whether `built` is there and no older than its sources."""
    if not os.path.exists(built):
        return False
    t = os.path.getmtime(built)
    return all(os.path.getmtime(s) <= t for s in made_of)


def torch_up_to_date() -> bool:
    """Whether the compiled binding is as good as it gets: built, tried in vain, or not wanted."""
    return torch_dir() is None or any(newer(f, torch_sources())
                                      for f in (torch_lib(), torch_lib() + ".failed"))


def up_to_date() -> bool:
    return newer(LIB, sources()) and torch_up_to_date()


def torch_dir():
    """The installed torch package's folder (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    where = list(spec.submodule_search_locations or []) if spec else []
    return where[0] if where else None


def torch_version() -> str:
    """The installed torch's version (read, not imported)."""
    try:
        with open(os.path.join(torch_dir(), "version.py")) as f:
            found = re.search(r"""^__version__[^=\n]*=\s*['"]([^'"\n]+)""", f.read(), re.M)
    except OSError:
        found = None
    return found.group(1) if found else "unknown"


def torch_lib() -> str:
    """The compiled binding for this Python and this torch: with others it is another file."""
    return os.path.join(LIBDIR, f"lm_torch.{sysconfig.get_config_var('SOABI')}.{torch_version()}.so")


def torch_command(out: str):
    """The compiler call for the compiled binding."""
    t = torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
            "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), os.path.join(CSRC, "lm_torch.cpp"), "-o", out,
            "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(t, "lib")]


def start(command):
    """A compiler at work beside the others, or the reason why it did not start."""
    try:
        return subprocess.Popen(command(), stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except (OSError, RuntimeError) as e:
        return str(e)


def finish(job):
    """(whether it succeeded, what it said)"""
    if isinstance(job, str):
        return False, job
    log = job.communicate()[0]
    return job.returncode == 0, log


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    library = force or not newer(LIB, sources())
    binding = torch_dir() is not None and (force or not torch_up_to_date())
    tmp = LIB + f".tmp{os.getpid()}"
    torch_tmp = LIB + f".torch.tmp{os.getpid()}"

    def compile_unit(unit, obj):
        return [nvcc(), *(extra or []), *(["-Xptxas=-v"] if verbose else []), *ARCH_FLAGS, "-O3",
                "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE,
                "-I", CSRC, "-c", "-o", obj, unit]

    # one object per source file, compiled side by side
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if library else []
    objs = [f"{tmp}.{os.path.basename(u)}.o" for u in units]
    try:
        torch_job = start(lambda: torch_command(torch_tmp)) if binding else None
        jobs = [start(lambda: compile_unit(u, o)) for u, o in zip(units, objs)]
        done = [finish(j) for j in jobs]
        if binding:
            ok, log = finish(torch_job)
            if verbose:
                sys.stderr.write(log)
            failed = torch_lib() + ".failed"
            if ok:
                os.replace(torch_tmp, torch_lib())
                if os.path.exists(failed):
                    os.remove(failed)
            else:
                if os.path.exists(torch_lib()):  # of other sources than the library's
                    os.remove(torch_lib())
                with open(failed, "w") as f:  # not tried again until a source or torch changes
                    f.write(log)
                warnings.warn("the compiled binding for torch tensors was not built; the 8-bit operators "
                              f"are marshalled in Python ({failed} has the compiler's words)",
                              RuntimeWarning, stacklevel=2)
        if library:
            if all(ok for ok, _ in done):
                done.append(finish(start(
                    lambda: [nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs])))
            failed = not all(ok for ok, _ in done)
            if failed or verbose:
                sys.stderr.write("".join(log for _, log in done))
            if failed:
                raise RuntimeError("nvcc failed building libvocoder.so")
            os.replace(tmp, LIB)
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
