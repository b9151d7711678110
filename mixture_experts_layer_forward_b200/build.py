"""Build the CUDA shared library (sm_100a) in-tree with nvcc.

The library has two translation units: csrc/moe_api.cu (the layer) and csrc/ops_api.cu (the
operators around it), which include the kernel headers; together they export the C ABI
declared in include/moe.h.
"""
from __future__ import annotations

import os
import shutil
import subprocess
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIB_PATH = PKG / "libmoe_b200.so"

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
]
UNITS = ("moe_api.cu", "ops_api.cu")


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh")) + [INCLUDE / "moe.h"]


def needs_build(out: Path = LIB_PATH) -> bool:
    if not out.exists():
        return True
    t = out.stat().st_mtime
    return any(s.stat().st_mtime > t for s in _sources())


def build_library(force: bool = False, out: Path = LIB_PATH, extra_flags=()) -> Path:
    """Compile the translation units (side by side) and link them into ``out`` (default: the
    in-tree libmoe_b200.so)."""
    out = Path(out)
    if not force and not needs_build(out):
        return out
    tag = f".tmp{os.getpid()}"
    tmp = out.with_name(out.name + tag)
    objs = [out.with_name(u + tag + ".o") for u in UNITS]
    common = [_nvcc(), *NVCC_FLAGS, *extra_flags, "-I", str(INCLUDE)]
    try:
        procs = [subprocess.Popen([*common, "-c", "-o", str(o), str(CSRC / u)])
                 for u, o in zip(UNITS, objs)]
        if any([p.wait() != 0 for p in procs]):
            raise RuntimeError("nvcc failed")
        subprocess.run([*common, "-shared", "-o", str(tmp), *map(str, objs)], check=True)
        os.replace(tmp, out)
    finally:
        for o in (*objs, tmp):
            o.unlink(missing_ok=True)
    return out


if __name__ == "__main__":
    print(build_library(force=True))
