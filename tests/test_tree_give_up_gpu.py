"""What the attention's tile kernel does when one of its bounded waits gives
up (tests/c/tree_give_up.cu, built with nvcc against the kernel's own source)."""
import os
import shutil
import subprocess

import pytest

from place_partial_rope_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc is not installed")
    exe = str(tmp_path_factory.mktemp("give_up") / "tree_give_up")
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", "-O3", "-I", build.INCLUDE, "-I", build.CSRC,
                    os.path.join(HERE, "c", "tree_give_up.cu"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("mode", ["agree", "fetch", "call"])
def test_give_up(program, mode):
    r = subprocess.run([program, mode], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout + r.stderr
