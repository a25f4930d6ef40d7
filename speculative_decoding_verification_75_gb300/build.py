"""Build ``lib/libspecverify.so`` (the CUDA verification library) in-tree.

Two translation units (the verification step, the paged KV cache), compiled
in parallel for sm_103a only and linked, and beside them ``lib/_svkv.so``, the
native module of ``kv.py`` (plain C++ against the installed PyTorch).  The
results are git-ignored; every machine that runs the library builds them from
source.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
SRC_DIR = PKG / "csrc"
MAIN = SRC_DIR / "spec_verify.cu"
PAGED_DIR = PKG / "paged"
UNITS = [MAIN, PAGED_DIR / "sv_paged.cu"]
INCLUDE = ROOT / "include"
LIB = PKG / "lib" / "libspecverify.so"
BINDING_SRC = PAGED_DIR / "sv_paged_binding.cpp"
BINDING = PKG / "lib" / "_svkv.so"

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
    if not LIB.exists() or not BINDING.exists():
        return True
    t = min(LIB.stat().st_mtime, BINDING.stat().st_mtime)
    return any(s.stat().st_mtime > t for s in [*sources(), BINDING_SRC])


def compile_command(unit: Path, out: Path, defines=()):
    return [nvcc(), *NVCC_FLAGS, *[f"-D{d}" for d in defines], f"-I{INCLUDE}", f"-I{SRC_DIR}",
            "-c", str(unit), "-o", str(out)]


def binding_command(out: Path):
    import torch
    root = Path(torch.__file__).resolve().parent
    cuda = Path(nvcc()).resolve().parents[1]
    includes = [INCLUDE, root / "include", root / "include" / "torch" / "csrc" / "api" / "include",
                sysconfig.get_paths()["include"], cuda / "include"]
    return ["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{i}" for i in includes], str(BINDING_SRC), f"-L{root / 'lib'}", "-ltorch_python",
            "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{root / 'lib'}", "-ldl",
            "-o", str(out)]


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
    binding = BINDING.with_name(f".{BINDING.name}.{tag}")

    def run(cmd):
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)

    try:
        jobs = [compile_command(u, o) for u, o in zip(UNITS, objects)] + [binding_command(binding)]
        with cf.ThreadPoolExecutor(len(jobs)) as ex:
            for f in [ex.submit(run, j) for j in jobs]:
                f.result()
        run(link_command(objects, tmp))
        os.replace(tmp, LIB)
        os.replace(binding, BINDING)
    finally:
        for o in objects:
            o.unlink(missing_ok=True)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
