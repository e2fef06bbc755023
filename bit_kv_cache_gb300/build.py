"""Builds libkvq.so (the C-ABI library) in-tree with nvcc for sm_103a.

    python bit_kv_cache_gb300/build.py [--force]

The translation units compile in parallel and link into
``bit_kv_cache_gb300/_build/libkvq.so``.  Nothing is installed outside the tree.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libkvq.so")
SOURCES = ["kvq_api.cu", "kvq_quant.cu", "kvq_decode.cu", "kvq_noalloc.cu", "kvq_paged.cu",
           "kvq_decode_paged.cu", "kvq_decode_rope.cu", "kvq_decode_nvfp4.cu", "kvq_selftest.cu",
           "kvq_chunk.cu", "kvq_chunk_attn.cu", "kvq_chunk_attn_block.cu", "kvq_chunk_combine.cu", "kvq_block.cu", "kvq_block_decode.cu",
           "kvq_append_rope.cu"]
HEADERS = ["kvq_device.cuh", "kvq_internal.h", "kvq_decode_fast.cuh", "kvq_host.h",
           "kvq_decode.cuh", "kvq_quantizer.cuh", "kvq_chunk.h",
           "kvq_chunk_attn.cuh", "kvq_chunk_attn_kernel.cuh", "kvq_tcgen05.cuh", "kvq_extend.cuh", "kvq_block.h", "kvq_block.cuh",
           "kvq_rope.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "kvq.h"),
                                                                 os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    objs = [os.path.join(BUILD, f.replace(".cu", ".o")) for f in SOURCES]

    def compile_one(i):
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, SOURCES[i]), "-o", objs[i]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (SOURCES[i], r.stdout, r.stderr))
        if verbose:
            sys.stdout.write(r.stdout + r.stderr)

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        list(ex.map(compile_one, range(len(SOURCES))))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
