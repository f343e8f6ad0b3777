"""Builds libpgd.so and libpgd_ext.so in-tree (paged_gqa_decode_gb300/_build/)
with nvcc for sm_103a.  Each .cu is compiled in parallel, then linked into the
library it belongs to, whose only exported symbols are the C ABI of
include/pgd.h or include/pgd_ext.h."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libpgd.so")
EXT_LIB = os.path.join(BUILD, "libpgd_ext.so")

SOURCES = ["pgd_api.cu", "kv_append.cu", "paged_decode_d64.cu", "paged_decode_d128.cu",
           "paged_prefill.cu", "paged_prefill_umma.cu", "paged_prefill_umma_d64.cu",
           "paged_prefill_pair.cu"]
EXT_SOURCES = ["pgd_ext_api.cu", "batch_ops.cu", "page_ops.cu", "shared_decode_d64.cu",
               "shared_decode_d128.cu", "mod_decode_d64.cu", "mod_decode_d128.cu",
               "mod_prefill.cu"] + [f"mod_prefill_d{d}_{kind}.cu" for d in (64, 128)
                                    for kind in ("mask", "cap", "bias", "cap_bias")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-Xptxas", "-v", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpgd")
    return path


def _inputs_newer_than(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
        os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    run = subprocess.run(cmd, capture_output=True, text=True)
    if run.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{run.stderr}")
    with open(os.path.join(BUILD, os.path.splitext(src)[0] + ".ptxas.txt"), "w") as f:
        f.write(run.stderr)
    return obj, run.stderr


def _link(target: str, objs: list[str]) -> None:
    tmp = target + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-Xlinker", "--exclude-libs,ALL", "-o", tmp, *objs]
    run = subprocess.run(cmd, capture_output=True, text=True)
    if run.returncode != 0:
        raise RuntimeError(f"link failed:\n{run.stderr}")
    os.replace(tmp, target)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compiles and links libpgd.so and libpgd_ext.so if any source is newer
    than one of them; returns libpgd.so's path."""
    os.makedirs(BUILD, exist_ok=True)
    if not force and not _inputs_newer_than(LIB) and not _inputs_newer_than(EXT_LIB):
        return LIB
    sources = SOURCES + EXT_SOURCES
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources)) as ex:
        results = list(ex.map(_compile, sources))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    _link(LIB, objs[:len(SOURCES)])
    _link(EXT_LIB, objs[len(SOURCES):])
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
