"""Build the CUDA library libeqlin.so in place (sm_100a only).

    python -m cyclic_group_dft_b200.build [--force] [--verbose]

nvcc cross-compiles for sm_100a without a GPU; the static CUDA runtime is
linked in, so the library loads on machines without a driver (it only needs
one to run).
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libeqlin.so")
OBJ = os.path.join(PKG, "_build")   # one object file, dependency list and command line per source

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _object_stale(obj: str, dep: str, made_by: str, command: str) -> bool:
    """Is the object older than its source, one of the headers it included, or this file, or was it made by another
    command (other flags, or another tree of which this one is a copy)?"""
    if not (os.path.exists(obj) and os.path.exists(dep) and os.path.exists(made_by)):
        return True
    with open(made_by) as f:
        if f.read() != command:
            return True
    t = os.path.getmtime(obj)
    with open(dep) as f:
        names = f.read().split(":", 1)[-1].replace("\\\n", " ").split()
    own = [n for n in names if os.path.abspath(n).startswith(ROOT)] + [os.path.abspath(__file__)]
    return any(not os.path.exists(n) or os.path.getmtime(n) > t for n in own)


def _compile(src: str, force: bool, verbose: bool, extra: list[str]) -> str:
    stem = os.path.join(OBJ, os.path.splitext(os.path.basename(src))[0])
    obj, dep, made_by = stem + ".o", stem + ".d", stem + ".cmd"
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src]
    if force or _object_stale(obj, dep, made_by, "\n".join(cmd)):
        tmp = f"{stem}.tmp{os.getpid()}"
        run = [*cmd, "-MD", "-MF", tmp + ".d", "-o", tmp + ".o"]
        if verbose:
            print(" ".join(run), file=sys.stderr)
        subprocess.run(run, check=True)
        if os.path.exists(made_by):
            os.remove(made_by)          # none while the object and its list are replaced
        os.replace(tmp + ".d", dep)
        os.replace(tmp + ".o", obj)
        with open(tmp + ".cmd", "w") as f:
            f.write("\n".join(cmd))
        os.replace(tmp + ".cmd", made_by)
    return obj


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile libeqlin.so unless it is newer than every source (sources in parallel, each
    only when it, a header that it includes or its command line changed)."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        objs = list(pool.map(lambda src: _compile(src, force, verbose, extra or []), sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv, extra=extra))
