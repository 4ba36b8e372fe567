"""In-tree build of libbf16delta.so and libbf16ops.so for GB300 (sm_103a).

Each CUDA translation unit is compiled in parallel with nvcc, then linked into its shared
library next to this file.  Only the symbols declared in include/*.h (libbf16delta) and
include/ops/*.h (libbf16ops) are exported.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbf16delta.so")
OPS_LIB = os.path.join(PKG, "libbf16ops.so")

SOURCES = ["bd_api.cu", "bd_encode.cu", "bd_scan.cu", "bd_apply.cu", "bd_checksum.cu",
           "bd_noalloc.cu"]
OPS_SOURCES = ["bo_adamw.cu", "bo_adapter.cu", "bo_adapter_tc.cu"]
LIBRARIES = {LIB: SOURCES, OPS_LIB: OPS_SOURCES}
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _inputs(lib: str = LIB) -> list[str]:
    """Every file that a library is built from."""
    prefix = "bo_" if lib == OPS_LIB else "bd_"
    files = [os.path.join(CSRC, s) for s in LIBRARIES[lib]]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC)
              if f.endswith(".cuh") and f.startswith(prefix)]
    dirs = [INCLUDE] + ([os.path.join(INCLUDE, "ops")] if lib == OPS_LIB else [])
    files += [os.path.join(d, f) for d in dirs for f in os.listdir(d) if f.endswith(".h")]
    return files


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs(lib))


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds each library that is missing or older than its sources; returns libbf16delta's
    path."""
    libs = [lib for lib in LIBRARIES if force or not up_to_date(lib)]
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs: dict[str, list[str]] = {lib: [] for lib in libs}
    for lib in libs:
        for src in LIBRARIES[lib]:
            obj = os.path.join(BUILD, src.replace(".cu", ".o"))
            objs[lib].append(obj)
            cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(f"{src}:\n{out.decode(errors='replace')}")
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    for lib in libs:
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs[lib]]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
