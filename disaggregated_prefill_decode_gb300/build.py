"""Builds libkvx.so in-tree with nvcc for sm_103a (one -gencode), translation units in parallel."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkvx.so")

SOURCES = ["kvx_plan.cpp", "kvx_tiles.cpp", "kvx_conn.cpp", "kvx_copy.cu", "kvx_push.cu", "kvx_match.cu", "kvx_cache.cpp",
           "kvx_slots.cu", "kvx_append.cu", "kvx_attend.cu", "kvx_attend_bf16.cu",
           "kvx_attend_f16.cu", "kvx_attend_e4m3_bf16.cu", "kvx_attend_e4m3_f16.cu", "kvx_latent.cu",
           "kvx_latent_tensor.cu", "kvx_page_calls.cpp", "kvx_pages.cu", "kvx_rotation.cpp",
           "kvx_rotate.cu", "kvx_shared_calls.cpp", "kvx_shared.cu", "kvx_shared_bf16.cu", "kvx_shared_f16.cu",
           "kvx_shared_e4m3_bf16.cu", "kvx_shared_e4m3_f16.cu", "kvx_rest_bf16.cu", "kvx_rest_f16.cu", "kvx_rest_e4m3_bf16.cu",
           "kvx_rest_e4m3_f16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input() -> float:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "kvx.h"), __file__]
    return max(os.path.getmtime(p) for p in deps)


def build(force: bool = False, verbose: bool = False, extra: tuple = ()) -> str:
    """Compile every translation unit and link libkvx.so (cudart linked statically). Skips the work
    when the library is newer than every source. Returns the library path."""
    if not force and not extra and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=PKG)
    os.close(fd)
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        os.unlink(tmp)
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    extra = tuple(a for a in sys.argv[1:] if a.startswith("-X"))
    print(build(force="--force" in sys.argv, verbose=True, extra=extra))
