"""Builds libzl_attn.so in-tree with nvcc for sm_103a.

    python -m mixed_length_dit_gb300.build [--force] [--verbose]

Each translation unit compiles in parallel into _build/, then one shared
library is linked next to this file.  A unit is recompiled when its source or
any header of csrc/ or include/ is newer than its object.  Beside them the
host compiler builds _bind.so (binding/bind.cpp, against PyTorch's headers),
the short way from tensors to the library.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libzl_attn.so")
BIND_SRC = os.path.join(PKG, "binding", "bind.cpp")
BIND = os.path.join(PKG, "_bind.so")
BIND_FOR = os.path.join(BUILD, "bind.torch")    # the version of PyTorch that _bind.so was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(obj, src, hdr_mtime):
    if not os.path.exists(obj):
        return True
    return os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_mtime)


def _torch_version():
    from importlib.metadata import version
    return version("torch")


def _bind_stale(hdr_mtime):
    """Sources newer than _bind.so, or another PyTorch than the one it was built for."""
    if _stale(BIND, BIND_SRC, hdr_mtime) or not os.path.exists(BIND_FOR):
        return True
    with open(BIND_FOR) as f:
        return f.read() != _torch_version()


def _bind_commands():
    """Compiles and links _bind.so, against the PyTorch that runs this."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(base, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cxx = shutil.which("g++") or "g++"
    obj = os.path.join(BUILD, "bind.cpp.o")
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             f'-DZL_TORCH_VERSION="{torch.__version__}"',
             *(f"-I{p}" for p in inc), "-c", BIND_SRC, "-o", obj],
            [cxx, "-shared", obj, "-o", BIND + ".tmp", "-L" + os.path.join(base, "lib"), "-L" + PKG, "-lzl_attn",
             "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])


def _link(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("link failed")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdr_mtime = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    cc = nvcc()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(obj, src, hdr_mtime):
            cmd = [cc, *ARCH, *COMMON, *extra_flags, "-c", src, "-o", obj]
            if src.endswith(".cu"):
                cmd[1:1] = ["-Xptxas", "-v"] if verbose else []
            jobs.append(cmd)
    units = len(jobs)
    bind_link = None
    if force or _bind_stale(hdr_mtime):
        compile_, bind_link = _bind_commands()
        jobs.insert(0, compile_)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        failed = [(c, r) for c, r in zip(jobs, results) if r.returncode != 0]
        for c, r in zip(jobs, results):
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(c) + "\n" + r.stdout + r.stderr)
        if failed:
            raise RuntimeError(f"the compiler failed for {len(failed)} unit(s)")
    if units or not os.path.exists(LIB) or force:
        tmp = LIB + ".tmp"
        _link([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"])
        os.replace(tmp, LIB)
    if bind_link:
        _link(bind_link)
        os.replace(BIND + ".tmp", BIND)
        with open(BIND_FOR, "w") as f:
            f.write(_torch_version())
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
