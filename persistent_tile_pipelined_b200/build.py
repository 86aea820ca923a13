"""Build the package's native libraries in-tree.

* ``synth/libtre_synth.so`` — the seeded input generator (gcc + OpenMP).
* ``libtre.so``             — the engine: host planner + C ABI (C++17), the
                              persistent sm_100a kernel and the prompt operators
                              (nvcc, -gencode arch=compute_100a,code=sm_100a).

Run ``python -m persistent_tile_pipelined_b200.build``.  nvcc cross-compiles without a
GPU, so this works on a CPU-only machine.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
ENGINE_LIB = os.path.join(PKG, "libtre.so")
SYNTH_LIB = os.path.join(PKG, "synth", "libtre_synth.so")

ENGINE_SOURCES = ["planner.cpp", "tre_api.cu", "engine.cu", "noalloc.cu",
                  "prompt_attention.cu", "mxfp4.cu", "mxfp4_matmul.cu", "add_rmsnorm.cu",
                  "ops_host.cu"]


def engine_headers():
    """Every header in csrc/: an edit to any of them rebuilds the library."""
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".h", ".cuh")))


NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the engine needs the CUDA toolkit to build")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _included(path: str, seen=None) -> list:
    """The headers of csrc/ and include/ that a source includes, directly or not."""
    seen = [] if seen is None else seen
    for name in re.findall(r'#include "([^"]+)"', open(path).read()):
        for folder in (CSRC, INCLUDE):
            p = os.path.join(folder, name)
            if os.path.exists(p) and p not in seen:
                seen.append(p)
                _included(p, seen)
    return seen


def build_synth(force: bool = False) -> str:
    src = os.path.join(PKG, "synth", "gen.c")
    if force or _stale(SYNTH_LIB, [src]):
        subprocess.check_call(["gcc", "-O2", "-fopenmp", "-fPIC", "-shared", "-std=c11", src,
                               "-o", SYNTH_LIB, "-lm"])
    return SYNTH_LIB


def _made_with(target: str, flags) -> bool:
    """Whether `target` was made with these flags, by the note beside it."""
    try:
        return open(target + ".flags").read() == "\n".join(flags)
    except OSError:
        return False


def _make(cmd, target: str, flags) -> None:
    """Run cmd, which makes `target`; the note of its flags is there only once it has."""
    note = target + ".flags"
    if os.path.exists(note):
        os.remove(note)
    subprocess.check_call(cmd)
    with open(note, "w") as f:
        f.write("\n".join(flags))


def build_engine(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    srcs = [os.path.join(CSRC, s) for s in ENGINE_SOURCES]
    deps = srcs + [os.path.join(CSRC, h) for h in engine_headers()] + [
        os.path.join(INCLUDE, "tre.h")]
    flags = [*NVCC_FLAGS, *extra_flags]
    objdir = os.path.join(PKG, "_build")
    linked = os.path.join(objdir, os.path.basename(ENGINE_LIB))  # its note stands with the objects
    if not (force or extra_flags or _stale(ENGINE_LIB, deps) or not _made_with(linked, flags)):
        return ENGINE_LIB
    nvcc = _nvcc()
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for s in srcs:
        obj = os.path.join(objdir, os.path.basename(s) + ".o")
        objs.append(obj)
        if not (force or extra_flags or _stale(obj, [s] + _included(s)) or
                not _made_with(obj, flags)):
            continue
        cmd = [nvcc, *flags, "-I", INCLUDE, "-I", CSRC, "-c", s, "-o", obj]
        if verbose and s.endswith(".cu"):
            cmd += ["-Xptxas", "-v"]
        _make(cmd, obj, flags)
    _make([nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", ENGINE_LIB,
           "-lcudart"], linked, flags)
    return ENGINE_LIB


def build_all(force: bool = False) -> None:
    build_synth(force)
    build_engine(force)


if __name__ == "__main__":
    build_all(force="--force" in sys.argv)
    print("built", ENGINE_LIB, SYNTH_LIB)
