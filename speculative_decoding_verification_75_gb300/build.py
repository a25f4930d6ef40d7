"""Build ``lib/libspecverify.so`` (the CUDA verification library) in-tree.

Two translation units (the verification step, the paged KV cache), compiled
in parallel for sm_103a only and linked.  The result is git-ignored; every
machine that runs the library builds it from source.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
SRC_DIR = PKG / "csrc"
MAIN = SRC_DIR / "spec_verify.cu"
PAGED_DIR = PKG / "paged"
UNITS = [MAIN, PAGED_DIR / "sv_paged.cu"]
INCLUDE = ROOT / "include"
LIB = PKG / "lib" / "libspecverify.so"

NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo",
              "-gencode", "arch=compute_103a,code=sm_103a",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify.so")


def sources():
    return [*UNITS, *sorted(SRC_DIR.glob("*.cuh")), *sorted(PAGED_DIR.glob("*.cuh")),
            *sorted(INCLUDE.glob("*.h"))]


def is_stale() -> bool:
    if not LIB.exists():
        return True
    t = LIB.stat().st_mtime
    return any(s.stat().st_mtime > t for s in sources())


def compile_command(unit: Path, out: Path, defines=()):
    return [nvcc(), *NVCC_FLAGS, *[f"-D{d}" for d in defines], f"-I{INCLUDE}", f"-I{SRC_DIR}",
            "-c", str(unit), "-o", str(out)]


def link_command(objects, out: Path):
    return [nvcc(), *NVCC_FLAGS, "-shared", *[str(o) for o in objects], "-o", str(out)]


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile the library if it is missing or older than its sources."""
    if not force and not is_stale():
        return LIB
    LIB.parent.mkdir(parents=True, exist_ok=True)
    tag = f"tmp{os.getpid()}"
    tmp = LIB.with_name(f".{LIB.name}.{tag}")
    objects = [LIB.parent / f".{u.stem}.{tag}.o" for u in UNITS]

    def run(cmd):
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)

    try:
        with cf.ThreadPoolExecutor(len(UNITS)) as ex:
            for f in [ex.submit(run, compile_command(u, o)) for u, o in zip(UNITS, objects)]:
                f.result()
        run(link_command(objects, tmp))
        os.replace(tmp, LIB)
    finally:
        for o in objects:
            o.unlink(missing_ok=True)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
