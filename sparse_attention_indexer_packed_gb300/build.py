"""Build libidx.so in-tree with nvcc for sm_103a.

The translation units compile in parallel into ``_build/`` and link into
``sparse_attention_indexer_packed_gb300/libidx.so`` with the CUDA runtime
linked statically, so the library loads without a driver (its symbols can be
inspected on a machine with no GPU).  ``_binding.so`` beside it is the CPython
module of the small-call operators (csrc/idx_binding.c); it needs gcc and Python's
headers, and where one is missing those operators go through ctypes.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libidx.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["idx_api.cu", "idx_score.cu", "idx_wide.cu", "idx_topk.cu", "idx_store.cu", "idx_noalloc.cu",
           "idx_attn.cu", "idx_attn4.cu", "idx_attn_wide.cu", "idx_kv.cu", "idx_norm.cu",
           "idx_rope.cu"]
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
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        elif r.stderr.strip():
            print(r.stderr.strip(), file=sys.stderr)     # warnings: registers that are spilled
        return r

    def compile_one(job):
        cmd, out = job
        run(cmd)
        os.replace(out + tag, out)

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        list(ex.map(compile_one, jobs))
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    relinked = force or jobs or _stale(LIB, objs)
    if relinked:
        tmp = LIB + tag
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if _build_binding([os.path.join(CSRC, "idx_binding.c"), headers[-1]], tag, run, force) or relinked:
        _drop_native_calls()
    return LIB


def _build_binding(deps: list, tag: str, run, force: bool) -> bool:
    """Build the CPython module from deps[0] where that is due and can be done.  True: the file
    changed."""
    if not force and not _stale(BINDING, deps):
        return False
    include = sysconfig.get_paths()["include"]
    missing = "gcc" if shutil.which("gcc") is None else (
        "" if os.path.exists(os.path.join(include, "Python.h")) else "Python.h")
    if missing:
        print(f"{missing} not found: the layer operators are called through ctypes", file=sys.stderr)
        if os.path.exists(BINDING):      # built from another state of the sources
            os.remove(BINDING)
            return True
        return False
    run(["gcc", "-O2", "-std=c11", "-Wall", "-fPIC", "-shared", "-I" + include, deps[0], "-o", BINDING + tag,
         "-L" + HERE, "-l:libidx.so", "-Wl,-rpath,$ORIGIN"])
    os.replace(BINDING + tag, BINDING)
    return True


def _drop_native_calls() -> None:
    """A process that has loaded the CPython module holds the library from before this build with
    it; its calls go through ctypes, to the library that lib() loads."""
    package = sys.modules.get("sparse_attention_indexer_packed_gb300")
    if package is not None and hasattr(package, "_lib"):
        for name in package._lib.NATIVE_CALLS:
            setattr(package, name, getattr(package._lib, name))


if __name__ == "__main__":
    print(build_library(verbose=True, force=True))
