"""Build libg4.so in-tree for sm_103a with nvcc (no cmake, no torch extension machinery).

    python -m accelerator_decode_gb300.build
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(HERE, "libg4.so")
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("g4.cu", "kv4.cu", "pages.cu", "attn16.cu")]
HEADERS = [os.path.join(HERE, "csrc", f) for f in (
    "common.cuh", "gemv.cuh", "gemv_s.cuh", "attn.cuh", "attn_mqa.cuh", "misc.cuh", "gemm_tc.cuh", "mega.cuh",
    "host.h", "mbar.cuh", "kv4_layout.h", "kv4_host.h", "kv4.cuh", "kv4_attend.cuh", "kv4_block.cuh",
    "tc05.cuh", "pages_layout.h", "pages.cuh", "paged_host.h", "attn16.cuh", "attn16_decode.cuh")]
HEADERS.append(os.path.join(os.path.dirname(HERE), "include", "g4.h"))
# the flags are in this file: an object older than it may have been compiled with others
DEPS = SOURCES + HEADERS + [os.path.abspath(__file__)]

NVCC_FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo",
              "-Xcompiler", "-fPIC"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _newer(target, deps):
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps if os.path.exists(p))


def up_to_date():
    return _newer(LIB, DEPS)


def build(force=False, verbose=False):
    """Compile the translation units in parallel, then link; an object newer than its source,
    every header and this file is kept."""
    if not force and up_to_date():
        return LIB
    jobs, objects = [], []
    for src in SOURCES:
        obj = os.path.join(HERE, os.path.basename(src)[:-3] + ".o")
        objects.append(obj)
        if not force and _newer(obj, [src] + [d for d in DEPS if d not in SOURCES]):
            continue
        cmd = [_nvcc()] + NVCC_FLAGS + ["-c", "-o", obj + ".tmp", src]
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append((subprocess.Popen(cmd), cmd, obj))
    failed = [cmd for p, cmd, _ in jobs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, obj in jobs:
        os.replace(obj + ".tmp", obj)
    tmp = LIB + ".tmp"
    cmd = [_nvcc()] + NVCC_FLAGS + ["-shared", "-o", tmp] + objects
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
