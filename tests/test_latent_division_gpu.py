"""How the attention over latent rows divides its work among blocks, a masked tile counted where it
lies (tests/c/latent_division.cu, built with nvcc against the kernel's own source)."""
import os
import shutil
import subprocess

import pytest

from place_partial_rope_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_division(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc is not installed")
    exe = str(tmp_path / "latent_division")
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", "-O3", "-I", build.INCLUDE, "-I", build.CSRC,
                    os.path.join(HERE, "c", "latent_division.cu"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout + r.stderr
