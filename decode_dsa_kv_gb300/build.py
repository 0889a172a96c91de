"""Build the CUDA library of the decode-step KV path for GB300 (sm_103a).

Every `csrc/*.cu` is compiled by nvcc in parallel, then linked into the
in-tree shared library `libdsakv.so` beside this file; `csrc/binding.cpp`, the
calls' Python entry points, becomes `_binding.so` beside it. Run as
`python -m decode_dsa_kv_gb300.build` or through `__graft_entry__.build()`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdsakv.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    deps = ([src] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + [os.path.join(INCLUDE, "dsakv.h")])
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps):
        return obj
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def _build_binding() -> None:
    src = os.path.join(CSRC, "binding.cpp")
    deps = (src, os.path.join(INCLUDE, "dsakv.h"), os.path.abspath(__file__))
    if (os.path.exists(BINDING)
            and os.path.getmtime(BINDING) >= max(os.path.getmtime(d) for d in deps)):
        return
    _run([nvcc(), "-O2", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I" + INCLUDE,
          "-I" + sysconfig.get_paths()["include"], "-shared", "-cudart", "shared", src, "-o",
          BINDING + ".tmp", "-L" + HERE, "-l:libdsakv.so", "-Xlinker", "-rpath,$ORIGIN"],
         "the binding failed")
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile and link libdsakv.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra or []), srcs))
    if (not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        _run([nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *objs], "link failed")
        os.replace(LIB + ".tmp", LIB)
        if verbose:
            print("built", LIB)
    _build_binding()
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
