"""Build ``lib/libspecverify.so`` (the CUDA verification library) in-tree.

Two translation units (the verification step, the paged KV cache), compiled
in parallel for sm_103a only and linked, and beside them ``lib/_svkv.*.so``,
the native module of ``kv.py`` (plain C++ against the installed PyTorch).  The
results are git-ignored; every machine that runs the library builds them from
source.  The library needs nvcc alone: where the module cannot be built (no g++,
no PyTorch headers) it is installed all the same.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
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


def binding_path() -> Path:
    """The native module for this Python and PyTorch, whose C++ interface
    differs from version to version."""
    import torch
    return LIB.with_name(f"_svkv.{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def _older(result: Path, inputs) -> bool:
    return not result.exists() or any(s.stat().st_mtime > result.stat().st_mtime for s in inputs)


def library_is_stale() -> bool:
    return _older(LIB, sources())


def binding_is_stale() -> bool:
    return _older(binding_path(), [BINDING_SRC, *INCLUDE.glob("*.h")])


def is_stale() -> bool:
    return library_is_stale() or binding_is_stale()


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


def _build_library(run, tag: str) -> None:
    tmp = LIB.with_name(f".{LIB.name}.{tag}")
    objects = [LIB.parent / f".{u.stem}.{tag}.o" for u in UNITS]
    try:
        with cf.ThreadPoolExecutor(len(UNITS)) as ex:
            for f in [ex.submit(run, compile_command(u, o)) for u, o in zip(UNITS, objects)]:
                f.result()
        run(link_command(objects, tmp))
        os.replace(tmp, LIB)
    finally:
        for o in objects:
            o.unlink(missing_ok=True)


def _build_binding(run, tag: str) -> None:
    path = binding_path()
    tmp = path.with_name(f".{path.name}.{tag}")
    try:
        run(binding_command(tmp))
        os.replace(tmp, path)
    except (OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"{path.name} could not be built, kv_write, kv_read, kv_compact and "
                      f"tree_attention are not available from Python: {e}")


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile what is missing or older than its sources."""
    LIB.parent.mkdir(parents=True, exist_ok=True)
    tag = f"tmp{os.getpid()}"

    def run(cmd):
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)

    jobs = [job for job, stale in ((_build_library, library_is_stale), (_build_binding, binding_is_stale))
            if force or stale()]
    with cf.ThreadPoolExecutor(2) as ex:
        for f in [ex.submit(job, run, tag) for job in jobs]:
            f.result()
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
