"""Build step: compiles csrc/*.cu for sm_100a into libmuse.so next to this file, and
csrc/binding.cpp (the CPython binding of the serving entry points) into _serving.so beside it.

Run as ``python -m clustered_softmax_attention_b200.build`` (or through
``__graft_entry__.build()``).  nvcc cross-compiles, so no GPU is needed.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libmuse.so")
BINDING = os.path.join(PKG, "_serving.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    nv = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nv):
        raise RuntimeError("nvcc not found")
    return nv


def _stale(obj: str, src: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(p) > t for p in [src, *deps])


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")))
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD_DIR, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or ptxas_info or _stale(o, s, deps):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or ptxas_info or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                failed.append(cmd[-3])
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    if jobs or not os.path.exists(OUT) or force:
        cmd = [nvcc, *ARCH, "-shared", "-o", OUT, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    _build_binding(verbose, force)
    return OUT


def _binding_made_for() -> str:
    """What _serving.so depends on besides its sources: an extension of another interpreter or torch
    does not load, or loads and breaks."""
    import torch

    return f"{sys.implementation.cache_tag} {sys.version} torch {torch.__version__} {torch.__file__}"


def _binding_stale() -> bool:
    stamp = os.path.join(BUILD_DIR, "binding.stamp")
    if _stale(BINDING, os.path.join(CSRC, "binding.cpp"), [os.path.join(ROOT, "include", "muse.h")]):
        return True
    if not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read() != _binding_made_for()


def _build_binding(verbose: bool, force: bool) -> None:
    """csrc/binding.cpp against this interpreter and its torch, linked to libmuse.so."""
    src = os.path.join(CSRC, "binding.cpp")
    if not force and not _binding_stale():
        return
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    dirs = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], *include_paths(),
            os.path.join(cuda, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in dirs), src, "-o", BINDING, *(f"-L{d}" for d in library_paths()),
           "-L" + PKG, "-l:libmuse.so", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("the binding did not build")
    with open(os.path.join(BUILD_DIR, "binding.stamp"), "w") as f:
        f.write(_binding_made_for())


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv, force="-f" in sys.argv)
    print(OUT)
