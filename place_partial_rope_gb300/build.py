"""Build ``librope_partial.so`` in-tree: nvcc for sm_103a, one process per
translation unit, then one link.  Run as ``python -m place_partial_rope_gb300.build``.

Flags: ``-O3 -lineinfo -gencode arch=compute_103a,code=sm_103a``; no
``--use_fast_math`` (it would change rounding); the kernels spell every
product and sum with the round-to-nearest intrinsics, so FMA contraction
cannot change their results either.  The CUDA runtime is linked statically,
so the library needs no libcudart at load time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "librope_partial.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]

CU_SOURCES = ["rope_kernels_bf16.cu", "rope_kernels_fp16.cu", "rope_kernels_fp32.cu",
              "rope_launch.cu", "rope_axes_bf16.cu", "rope_axes_fp16.cu", "rope_axes_fp32.cu",
              "rope_axes_launch.cu", "rope_cache_bf16.cu", "rope_cache_fp16.cu",
              "rope_cache_fp32.cu", "rope_cache_launch.cu", "rope_tree_bf16.cu",
              "rope_tree_fp16.cu", "rope_tree_fp8.cu", "rope_tree_int8.cu", "rope_tile_bf16.cu",
              "rope_tile_fp16.cu", "rope_tile_fp8.cu", "rope_tile_int8.cu", "rope_tree_launch.cu"]
CPP_SOURCES = ["rope_host.cpp", "rope_serving_host.cpp"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librope_partial.so")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    common = ["-std=c++17", "-O3", "-I", INCLUDE, "-I", CSRC]
    jobs = []
    for src in CU_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc, *ARCH, "-lineinfo", *common, "-Xcompiler", "-fPIC", "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append((cmd, obj))
    for src in CPP_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc, *common, "-Xcompiler", "-fPIC,-Wall", "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((cmd, obj))

    def run(job):
        cmd, _ = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        results = list(ex.map(run, jobs))
    for cmd, r in results:
        if verbose_ptxas and r.stderr:
            sys.stderr.write(r.stderr)
        if r.returncode != 0:
            raise RuntimeError("compile failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    tmp = LIB + ".tmp"
    link = [nvcc, *ARCH, "-shared", "-o", tmp] + [obj for _, obj in jobs]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + " ".join(link) + "\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas-v" in sys.argv))
