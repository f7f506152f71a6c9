"""Build the sm_100a shared library libpe.so in-tree with nvcc (no GPU needed).

`--debug-bounds` builds libpe_debug.so instead: the same sources with
-DPE_DEBUG_BOUNDS, whose kernels check every data-dependent global access
against the buffer it indexes and report PE_ERR_DEVICE_BOUNDS instead of
touching memory outside it.  Load it by setting PE_LIB to its path before
importing the package."""
from __future__ import annotations

import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpe.so")
DEBUG_LIB = os.path.join(HERE, "libpe_debug.so")
SOURCES = [os.path.join(CSRC, "pe_api.cu"), os.path.join(CSRC, "pe_tower.cu")]
OBJ_DIR = os.path.join(HERE, "_build")    # one object per source and variant, reused while its inputs are older
# every file the build reads: a change to any of them makes the library stale
DEPS = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))) + \
    [os.path.join(os.path.dirname(HERE), "include", "pe.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-v",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in DEPS)


def inputs(path: str) -> set:
    """`path` and every file it includes by a quoted name, directly or not."""
    seen, todo = set(), [os.path.normpath(path)]
    while todo:
        f = todo.pop()
        if f not in seen:
            seen.add(f)
            with open(f, encoding="utf-8") as src:
                names = re.findall(r'^\s*#\s*include\s+"([^"]+)"', src.read(), flags=re.M)
            todo += [os.path.normpath(os.path.join(os.path.dirname(f), n)) for n in names]
    return seen


def _run(cmd, what: str, verbose: bool) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc failed building {what}")
    if verbose:
        sys.stderr.write(r.stderr)


def _object(src: str, suffix: str, extra, force: bool, verbose: bool) -> str:
    obj = os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(src))[0] + suffix + ".o")
    newest = max(os.path.getmtime(f) for f in inputs(src) | {os.path.abspath(__file__)})
    if force or not os.path.exists(obj) or os.path.getmtime(obj) < newest:
        tmp = f"{obj}.tmp{os.getpid()}.o"
        flags = [f for f in NVCC_FLAGS if f != "-shared"]
        _run([nvcc(), *flags, *extra, "-c", src, "-o", tmp], os.path.basename(obj), verbose)
        os.replace(tmp, obj)
    return obj


def build(force: bool = False, verbose: bool = False, debug_bounds: bool = False) -> str:
    lib = DEBUG_LIB if debug_bounds else LIB
    if not force and not stale(lib):
        return lib
    os.makedirs(OBJ_DIR, exist_ok=True)
    extra = ["-DPE_DEBUG_BOUNDS"] if debug_bounds else []
    suffix = "_debug" if debug_bounds else ""
    with ThreadPoolExecutor(len(SOURCES)) as pool:   # the sources compile side by side
        objs = list(pool.map(lambda s: _object(s, suffix, extra, force, verbose), SOURCES))
    tmp = lib + f".tmp{os.getpid()}"
    _run([nvcc(), *NVCC_FLAGS, *objs, "-o", tmp], os.path.basename(lib), verbose)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug_bounds="--debug-bounds" in sys.argv))
