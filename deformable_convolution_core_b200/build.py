"""Build the CUDA library in-tree: libdcncore.so next to this file.

nvcc compiles the translation units of csrc/ (dcn_core.cu: the core operator,
its guide branch and projection; dcn_linear_fp8.cu: the e4m3 quantiser and
linear layer; dcn_block_norm.cu: the block's norms) for sm_100a only (the
library has no other target) with the C ABI of include/dcn_core.h, side by side, and links them.
Fast-math is deliberately off: the softmax uses expf and the sampling
location must be rounded exactly as the operator's contract states.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdcncore.so")
# The bounds-checked build: every global access of the kernels is tested
# against its tensor's extent first (a substitute for a memory checker).
LIB_CHECKED = os.path.join(HERE, "libdcncore_checked.so")
SOURCES = [os.path.join(CSRC, f) for f in ("dcn_core.cu", "dcn_linear_fp8.cu", "dcn_block_norm.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
                  if f.endswith((".cuh", ".h"))] + [os.path.join(INCLUDE, "dcn_core.h")]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def object_path(source: str, checked: bool = False) -> str:
    name = os.path.splitext(os.path.basename(source))[0]
    return os.path.join(HERE, "build", name + ("_checked.o" if checked else ".o"))


def headers_of(source: str, seen: set[str] | None = None) -> set[str]:
    """The source and every header of the library it includes, directly or not."""
    seen = set() if seen is None else seen
    seen.add(source)
    with open(source) as f:
        for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
            for folder in (CSRC, INCLUDE):
                path = os.path.join(folder, name)
                if os.path.exists(path) and path not in seen:
                    headers_of(path, seen)
    return seen


def compile_command(source: str, out: str, extra: list[str] | None = None) -> list[str]:
    return [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
            "-std=c++17", "-c", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
            "-I", INCLUDE, "-o", out] + (extra or []) + [source]


def link_command(objects: list[str], out: str) -> list[str]:
    return [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", out] + objects


def run_nvcc(command: list[str]) -> str:
    res = subprocess.run(command, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    return res.stderr


def compile_object(source: str, force: bool, verbose: bool, checked: bool) -> str:
    """Compile one translation unit if it, or a header it includes, is newer than its object."""
    obj = object_path(source, checked)
    if not force and os.path.exists(obj):
        t = os.path.getmtime(obj)
        if all(os.path.getmtime(d) <= t for d in headers_of(source)):
            return obj
    os.makedirs(os.path.dirname(obj), exist_ok=True)
    tmp = obj + ".tmp.%d" % os.getpid()
    extra = (["-Xptxas", "-v"] if verbose else []) + (["-DDCN_CHECK_BOUNDS"] if checked else [])
    out = run_nvcc(compile_command(source, tmp, extra))
    if verbose:
        sys.stderr.write(out)
    os.replace(tmp, obj)
    return obj


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in DEPS)


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Build libdcncore.so (or, with checked=True, libdcncore_checked.so with
    -DDCN_CHECK_BOUNDS) next to this file, if a source is newer."""
    lib = LIB_CHECKED if checked else LIB
    if force or needs_build(lib):
        with ThreadPoolExecutor(len(SOURCES)) as ex:
            objects = list(ex.map(lambda src: compile_object(src, force, verbose, checked), SOURCES))
        tmp = lib + ".tmp.%d" % os.getpid()
        run_nvcc(link_command(objects, tmp))
        os.replace(tmp, lib)
    return lib


def build_all(force: bool = False) -> list[str]:
    """Build the library and its bounds-checked twin side by side."""
    with ThreadPoolExecutor(2) as ex:
        jobs = [ex.submit(build, force, False, c) for c in (False, True)]
        return [j.result() for j in jobs]


if __name__ == "__main__":
    if "--all" in sys.argv:
        print(build_all(force="--force" in sys.argv))
    else:
        print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                    checked="--checked" in sys.argv))
