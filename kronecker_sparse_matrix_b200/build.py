"""Builds the KS CUDA library in-tree: kronecker_sparse_matrix_b200/libks_b200.so,
and, where torch is installed, the host-side module that reads tensors for it,
_ks_marshal (with the interpreter's suffix).  The library needs neither torch nor Python.

Every kernel is compiled for sm_100a only
(``-gencode arch=compute_100a,code=sm_100a``) with nvcc; objects go to
``_build/`` at the repository root.  Usage: ``python -m
kronecker_sparse_matrix_b200.build [--force] [--verbose]``, or this file as a script
where there is no torch.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libks_b200.so")
MARSHAL_SRC = os.path.join(CSRC, "ks_marshal.cpp")
MARSHAL = os.path.join(PKG, "_ks_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
MARSHAL_STAMP = os.path.join(BUILD, "_ks_marshal.stamp")  # what the module was built for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KS library needs the CUDA toolkit to build")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _newest(paths):
    return max((os.path.getmtime(p) for p in paths), default=0.0)


def _compile(src: str, obj: str, verbose: bool) -> str:
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(-4, "-Xptxas")
        cmd.insert(-4, "-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return (r.stdout + r.stderr).strip()


def build_marshal(force: bool = False) -> Optional[str]:
    """The CPython module that reads tensors (host code only); None without torch, whose
    headers it needs.  Rebuilt when its source, Python or torch has changed."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    include = os.path.join(os.path.dirname(spec.origin), "include")
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # (a source tree on the path)
        version = "unknown"
    stamp = f"python {sys.version}\ntorch {version} {include}\n"
    if not force and os.path.exists(MARSHAL) and os.path.exists(MARSHAL_STAMP):
        read = (MARSHAL_SRC, os.path.join(INCLUDE, "ks.h"), os.path.join(include, "ATen", "dlpack.h"))
        newest = _newest([p for p in read if os.path.exists(p)])
        with open(MARSHAL_STAMP) as f:
            if f.read() == stamp and os.path.getmtime(MARSHAL) >= newest:
                return MARSHAL
    os.makedirs(BUILD, exist_ok=True)
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-o", tmp, MARSHAL_SRC,
           "-I", sysconfig.get_paths()["include"], "-I", INCLUDE, "-I", include]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on ks_marshal.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_STAMP, "w") as f:
        f.write(stamp)
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdr_time = _newest(headers())
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time):
            jobs.append((src, obj))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = {ex.submit(_compile, s, o, verbose): s for s, o in jobs}
            for fut in cf.as_completed(futs):
                out = fut.result()
                if verbose and out:
                    print(f"== {os.path.basename(futs[fut])}\n{out}", file=sys.stderr)
    if force or jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest(objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    build_marshal(force)  # after the library, which does not need it
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
