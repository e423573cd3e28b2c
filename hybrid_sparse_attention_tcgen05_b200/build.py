"""Build libhysparse.so in-tree for B200 (sm_100a) with nvcc.

    python -m hybrid_sparse_attention_tcgen05_b200.build [--force] [--verbose-ptxas]

Each ``csrc/*.cu`` compiles to ``_build/<name>.o`` (in parallel, only when
stale), then everything links into ``hybrid_sparse_attention_tcgen05_b200/
libhysparse.so`` with the CUDA runtime linked statically.  ``csrc/binding.cpp``
becomes ``_binding.so``, the native half of ragged.py, against the torch that
is installed.
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libhysparse.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(f) for f in files), default=0.0)


def _compile(src: str, obj: str, ptxas_verbose: bool) -> str:
    cmd = [nvcc(), *ARCH, *CFLAGS, "-c", src, "-o", obj]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{res.stderr}")
    return res.stderr


def _build_binding() -> None:
    import sysconfig

    import torch

    t = os.path.dirname(torch.__file__)
    tmp = BINDING + f".tmp{os.getpid()}"
    # the g++ that nvcc uses too (not $CXX): one that links its own libstdc++
    # statically crashes where torch's headers format a message
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           "-isystem", f"{t}/include", "-isystem", f"{t}/include/torch/csrc/api/include",
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           f"-L{t}/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for binding.cpp:\n{res.stderr}")
    os.replace(tmp, BINDING)


def _binding_stale() -> bool:
    if not os.path.exists(BINDING):
        return True
    import torch

    newest = max(os.path.getmtime(f) for f in (os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "hysparse.h"),
                                               os.path.join(os.path.dirname(torch.__file__), "version.py")))
    return os.path.getmtime(BINDING) < newest


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    dep_t = _deps_mtime()
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or ptxas_verbose or not os.path.exists(obj) or \
                os.path.getmtime(obj) < max(os.path.getmtime(src), dep_t):
            jobs.append((src, obj))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            futs = {ex.submit(_compile, s, o, ptxas_verbose): s for s, o in jobs}
            for f in cf.as_completed(futs):
                msg = f.result()
                if msg and (ptxas_verbose or not quiet):
                    sys.stderr.write(f"== {os.path.basename(futs[f])}\n{msg}")
    if jobs or force or not os.path.exists(LIB) or \
            os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        res = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs],
                             capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        os.replace(tmp, LIB)
    # last: it needs torch's and Python's headers, which callers of the C library may lack
    if force or _binding_stale():
        _build_binding()
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas, quiet=False))
