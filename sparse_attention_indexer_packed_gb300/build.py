"""Build libidx.so in-tree with nvcc for sm_103a.

The translation units compile in parallel into ``_build/`` and link into
``sparse_attention_indexer_packed_gb300/libidx.so`` with the CUDA runtime
linked statically, so the library loads without a driver (its symbols can be
inspected on a machine with no GPU).  ``_binding.so`` beside it is the CPython
module of the small-call operators (csrc/idx_binding.c).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libidx.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["idx_api.cu", "idx_score.cu", "idx_wide.cu", "idx_topk.cu", "idx_store.cu", "idx_noalloc.cu",
           "idx_attn.cu", "idx_attn_wide.cu", "idx_kv.cu", "idx_norm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _stale(out: str, deps: list) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build_library(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(HERE, "..", "include", "idx.h"))
    # every output is written under a name of this process's own and then
    # renamed into place, so builders running at once (one per rank of a
    # multi-GPU run) never read or link a half-written file
    tag = f".{os.getpid()}.tmp"
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or _stale(o, [s] + headers):
            jobs.append(([nvcc, *ARCH, *FLAGS, "-c", s, "-o", o + tag], o))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        return r

    def compile_one(job):
        cmd, out = job
        run(cmd)
        os.replace(out + tag, out)

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        list(ex.map(compile_one, jobs))
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + tag
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    src = os.path.join(CSRC, "idx_binding.c")
    if force or _stale(BINDING, [src, headers[-1]]):
        tmp = BINDING + tag
        run(["gcc", "-O2", "-std=c11", "-Wall", "-fPIC", "-shared", "-I" + sysconfig.get_paths()["include"],
             src, "-o", tmp, "-L" + HERE, "-l:libidx.so", "-Wl,-rpath,$ORIGIN"])
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build_library(verbose=True, force=True))
