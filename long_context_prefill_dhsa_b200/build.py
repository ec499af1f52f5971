"""Build libdhsa.so (the C-ABI library) in-tree with nvcc for sm_100a, and
the Python binding's argument checks (csrc/marshal.cpp) with g++.

    python -m long_context_prefill_dhsa_b200.build [--verbose-ptxas] [--force]

Objects go to long_context_prefill_dhsa_b200/_build/, the shared libraries
next to this file. A rebuild happens only when a source or header is newer
than the libraries (or with --force). The library needs nvcc alone, and is
built whatever becomes of the checks; those read tensors in torch's own layout,
so their file's name says for which torch and Python they were built, and no
other opens it. Without torch they are not built.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdhsa.so")
HEADER = os.path.join(ROOT, "include", "dhsa.h")
SOURCES = ["abi.cu", "pool.cu", "score_topk.cu", "csr.cu", "items.cu", "attn.cu", "attn_fwd.cu", "attn_short.cu",
           "rotary.cu", "tree_attn.cu", "tree_weight.cu", "tree_join.cu", "evict.cu"]
HEADERS = ["common.cuh", "sm100_ptx.cuh", "tmap.cuh", "pool_row.cuh", "cache.cuh",
           "tree.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def marshal_path() -> str:
    """Where the binding's compiled checks for this torch and Python are."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:      # run from its source tree, say
        from torch import __version__ as torch
    return os.path.join(PKG, f"_marshal-torch{torch}-{sysconfig.get_config_var('SOABI')}.so")


def _newer_than(path: str, files) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in files)


def library_up_to_date() -> bool:
    return _newer_than(LIB, [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [HEADER])


def marshal_up_to_date() -> bool:
    return _newer_than(marshal_path(), [os.path.join(CSRC, "marshal.cpp"), HEADER])


def build_library(verbose_ptxas: bool = False):
    os.makedirs(OBJ, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
                    "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OBJ, src.replace(".cu", ".o"))
        cmd = [nvcc()] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for src, _, r in results:
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose_ptxas and r.stderr:
            sys.stderr.write(r.stderr)
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for _, o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def build_marshal():
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    path = marshal_path()
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-o", tmp, os.path.join(CSRC, "marshal.cpp")]
    for d in (os.path.join(ROOT, "include"), os.path.join(torch, "include"),
              os.path.join(torch, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
              os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")):
        cmd += ["-I", d]
    cmd += ["-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Builds what is not up to date. A failure of the checks is raised after
    the library is in place."""
    def checks():
        if importlib.util.find_spec("torch") is not None and (force or not marshal_up_to_date()):
            build_marshal()

    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        marshal = ex.submit(checks)
        if force or not library_up_to_date():
            build_library(verbose_ptxas)
        marshal.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv))
