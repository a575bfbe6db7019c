"""Build libtreeverify.so (nvcc, sm_100a) and _paged.so, the binding of the
paged calls (g++, against the installed torch), in-tree.

    python -m tree_verification_verify_b200.build
"""

from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtreeverify.so")
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "--threads", "0",
]


BINDING = os.path.join(HERE, "_paged.so")
BINDING_SRC = os.path.join(CSRC, "paged_binding.cpp")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(f) > t for f in deps)


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def binding_against() -> str:
    """The torch and Python whose binary interfaces the binding uses."""
    import torch
    return f"torch {torch.__version__} python {sysconfig.get_config_var('SOABI')}"


def binding_built_against() -> str:
    """What the binding says it was built against (its source has the text as a string); empty: nothing."""
    if not os.path.exists(BINDING):
        return ""
    with open(BINDING, "rb") as f:
        found = re.search(rb"tv_paged built against ([^;]*);", f.read())
    return found.group(1).decode() if found else ""


def _binding_stale() -> bool:
    return _older(BINDING, [BINDING_SRC] + _headers()) or binding_built_against() != binding_against()


def binding_command(out: str):
    """g++ command of the binding."""
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(shutil.which(os.environ.get("NVCC", "nvcc")) or "/usr/local/cuda/bin/nvcc"))
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DTV_BUILT_AGAINST="tv_paged built against {binding_against()};"'] + [f"-I{i}" for i in inc] + \
        [BINDING_SRC, "-o", out, "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
         "-lc10_cuda", "-L" + os.path.join(cuda, "lib64"), "-lcudart"]


def _run(jobs, verbose: bool):
    """The commands of (output, command), at the same time; each output that was made is put in place.  Returns the
    errors by output, when all have ended."""
    procs, errors = [], {}
    for out, cmd in jobs:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        try:
            procs.append((out, cmd, subprocess.Popen(cmd)))
        except OSError as e:
            errors[out] = e
    for out, cmd, p in procs:
        if p.wait() != 0:
            errors[out] = subprocess.CalledProcessError(p.returncode, cmd)
        else:
            os.replace(out + ".tmp", out)
    return errors


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA sources into one shared library, and the binding
    (each skipped when up to date).  Returns the library path.  The library
    stands by itself: without a C++ compiler or Python's headers the binding
    is left out with a warning, and the paged calls of the package say so."""
    nvcc = os.environ.get("NVCC", "nvcc")
    jobs = []
    if force or _stale():
        jobs.append((LIB, [nvcc] + NVCC_FLAGS + ["-I", os.path.join(ROOT, "include")] + sources() + ["-o", LIB + ".tmp"]))
    if force or _binding_stale():
        jobs.append((BINDING, binding_command(BINDING + ".tmp")))
    errors = _run(jobs, verbose)
    if LIB in errors:
        raise errors[LIB]
    if BINDING in errors:
        warnings.warn(f"the binding of the paged calls was not built ({errors[BINDING]}); {LIB} was")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
