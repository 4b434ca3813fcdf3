"""Build libkvd.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc.

Each translation unit is compiled in parallel, then linked into one shared
library under ``paged_gqa_decode_kvd_gb300/_build/``.  No CPU code path exists:
the library is the product.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libkvd.so")
SOURCES = ["kvd_api.cu", "kvd_append.cu", "kvd_decode.cu", "kvd_decode_lowbit.cu", "kvd_combine.cu", "kvd_noalloc.cu",
           "kvd_tier.cu", "kvd_measure.cu", "kvd_rope.cu", "kvd_chunk.cu",
           "kvd_chunk_lowbit.cu", "kvd_compact.cu", "kvd_latent_api.cu", "kvd_latent_cache.cu", "kvd_latent_attn.cu",
           "kvd_latent_prefill.cu"]
HEADERS = ["kvd_common.cuh", "kvd_internal.h", "kvd_decode_kernel.cuh", "kvd_chunk.h", "kvd_tcgen.cuh",
           "kvd_chunk_kernel.cuh", "kvd_pool.h", "kvd_latent.h", os.path.join("..", "..", "include", "kvd.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvd.so")
    return path


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS]
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc(), "-c", *ARCH, *FLAGS, "-o", o, s]
            if verbose:
                cmd.insert(2, "-Xptxas=-v")
            jobs.append(cmd)
    with cf.ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
        for r in ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs):
            if r.returncode != 0:
                raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
            if verbose and r.stderr:
                print(r.stderr)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc(), "-shared", *ARCH, "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
