"""Build ``libspec_verify.so`` and ``libspec_cache.so`` (the C-ABI libraries) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libspec_verify.so")
CACHE_LIB = os.path.join(HERE, "libspec_cache.so")
HEADER = os.path.join(ROOT, "include", "spec_verify.h")


def _csrc(*names):
    return [os.path.join(CSRC, f) for f in names]


SOURCES = _csrc("spec_verify.cu")
DEPS = SOURCES + _csrc("sv_common.cuh", "sv_rows.cuh", "sv_seq.cuh", "sv_resid.cuh", "sv_ptx.cuh", "sv_procs.cuh",
                       "sv_nucleus.cuh", "sv_tree.cuh", "sv_head.cuh") + [HEADER]
CACHE_SOURCES = _csrc("spec_cache.cu")
CACHE_DEPS = CACHE_SOURCES + _csrc("sc_common.cuh", "sc_attend.cuh", "sc_store.cuh", "sv_ptx.cuh") + [
    HEADER, os.path.join(ROOT, "include", "spec_cache.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xcompiler", "-fvisibility=hidden",
]


def nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def up_to_date(lib: str = LIB, deps=None) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in (DEPS if deps is None else deps))


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date; returns the path of ``libspec_verify.so``."""
    running = []
    for lib, sources, deps in ((LIB, SOURCES, DEPS), (CACHE_LIB, CACHE_SOURCES, CACHE_DEPS)):
        if not force and up_to_date(lib, deps):
            continue
        cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-o", lib + ".tmp"] + sources
        running.append((lib, subprocess.Popen(cmd)))
    if any([p.wait() for _, p in running]):
        raise RuntimeError("nvcc failed")
    for lib, _ in running:
        os.replace(lib + ".tmp", lib)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose="-v" in sys.argv))
