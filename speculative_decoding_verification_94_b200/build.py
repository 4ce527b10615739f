"""Build libsv.so (the CUDA library) in-tree for sm_100a with nvcc, and the
native part of its Python binding with the host compiler."""
from __future__ import annotations

import os
import subprocess
import sys
from importlib import metadata
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
SOURCES = ["sv_api.cu", "sv_chain_bf16.cu", "sv_chain_f32.cu", "sv_kv.cu"]
LIB = PKG / "libsv.so"
BIND = PKG / "_svkv.so"  # Python module over libsv.so, for the paged cache calls
BOUND = PKG / "_build" / "_svkv.txt"  # the torch and Python it was built for
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden"]


def _bound_to() -> str:
    """What the native half of the binding is compiled against."""
    return f"torch {metadata.version('torch')}, {sys.implementation.cache_tag}"


def _stale() -> bool:
    if not LIB.exists() or not BIND.exists():
        return True
    if not BOUND.exists() or BOUND.read_text() != _bound_to():
        return True
    t = min(LIB.stat().st_mtime, BIND.stat().st_mtime)
    deps = list(CSRC.glob("*")) + [PKG.parent / "include" / "sv.h", Path(__file__)]
    return any(d.stat().st_mtime > t for d in deps if d.exists())


def _bind_command(obj: Path) -> list:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import CUDA_HOME, include_paths
    inc = [*include_paths(), sysconfig.get_paths()["include"],
           os.path.join(CUDA_HOME or "/usr/local/cuda", "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-isystem{d}" for d in inc], "-c", str(CSRC / "sv_bind.cpp"), "-o", str(obj)]


def build(force: bool = False, verbose: bool = False, jobs: int = 4) -> Path:
    if not force and not _stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    objdir = PKG / "_build"
    objdir.mkdir(exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = objdir / (src + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH, *FLAGS, "-c", str(CSRC / src), "-o", str(obj)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    tmp_bind = BIND.with_suffix(f".{os.getpid()}.tmp")
    procs.append(("sv_bind.cpp", subprocess.Popen(_bind_command(objdir / "sv_bind.o"),
                                                  stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stderr.write(out.decode())
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = LIB.with_suffix(f".{os.getpid()}.tmp")
    subprocess.run([nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *map(str, objs), "-o", str(tmp)],
                   check=True)
    os.replace(tmp, LIB)
    from torch.utils.cpp_extension import library_paths
    libs = [f"-L{d}" for d in library_paths()]
    subprocess.run([os.environ.get("CXX", "g++"), "-shared", str(objdir / "sv_bind.o"), "-o",
                    str(tmp_bind), f"-L{PKG}", "-l:libsv.so", "-Wl,-rpath,$ORIGIN", *libs, "-lc10",
                    "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], check=True)
    BOUND.write_text(_bound_to())
    os.replace(tmp_bind, BIND)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
