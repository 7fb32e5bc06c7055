"""Compile libgla.so (the CUDA kernels + C ABI) for sm_103a with nvcc, in-tree.

Each translation unit is compiled in parallel; the shared library links the CUDA runtime
statically, so it depends only on the driver (libcuda) at run time, loaded lazily by the
runtime.  The result goes to gated_linear_attention_chunked_gb300/_lib/libgla.so.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libgla.so")

SOURCES = ["api.cu", "decode.cu", "convert.cu", "chunk_fwd.cu", "chunk_bwd.cu", "noalloc.cu", "seg_scan.cu", "head_norm.cu", "conv.cu",
           "api_layer.cu", "gated_scan.cu", "layer_norm.cu",
           "window_fwd.cu", "window_bwd.cu", "window_decode.cu",
           "api_serving.cu", "rotary.cu", "window_cache8.cu", "window_decode8.cu", "window_chunk.cu",
           "window_chunk8.cu"]
HEADERS = ["ptx.cuh", "tmap.h", "kernels.h", "scan_common.cuh", "elem.cuh",
           "gated_scan.h", "layer_norm.h", "window_attn.h", "mma.cuh", "window_common.cuh",
           "window_wait.cuh", "api_checks.h", "rotary.h", "window_serve.h", "code8.cuh",
           "window_packed.cuh", "window_chunk.cuh", "window_rows8.cuh", "window_join.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgla")


def _digest() -> str:
    h = hashlib.sha256()
    h.update(" ".join(NVCC_FLAGS).encode())
    for f in SOURCES + HEADERS:
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + fh.read())
    with open(os.path.join(INCLUDE, "gla.h"), "rb") as fh:
        h.update(fh.read())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libgla.so unless an up-to-date one exists; returns its path."""
    digest = _digest()
    stamp = os.path.join(OUT_DIR, "libgla.stamp")
    if not force and os.path.exists(LIB) and os.path.exists(stamp):
        with open(stamp) as fh:
            if fh.read().strip() == digest:
                return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [cc] + NVCC_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([cc] + ARCH + ["-shared", "-o", tmp] + objs)
    os.replace(tmp, LIB)
    with open(stamp, "w") as fh:
        fh.write(digest)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
