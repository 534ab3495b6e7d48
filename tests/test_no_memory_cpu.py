"""Host memory that runs out inside the library ends in an error status
(tests/c/tree_no_memory.cpp, with a stand-in for the CUDA runtime; no GPU)."""
import os
import shutil
import subprocess

import pytest

from place_partial_rope_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_exception_reaches_a_c_caller(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    gxx = shutil.which("g++")
    if not os.path.exists(nvcc) or not gxx:
        pytest.skip("nvcc or g++ is not installed")
    flags = ["-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC]
    objects = []
    for src in ("rope_tree_launch.cu", "rope_launch.cu"):
        objects.append(str(tmp_path / (src + ".o")))
        subprocess.run([nvcc, *build.ARCH, *flags, "-c", os.path.join(build.CSRC, src), "-o", objects[-1]], check=True)
    exe = str(tmp_path / "no_memory")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    subprocess.run([gxx, *flags, "-I", cuda, os.path.join(HERE, "c", "tree_no_memory.cpp"), *objects, "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout + r.stderr
