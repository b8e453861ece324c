"""The experts' kernels run on the host, a fiber for each lane, in orders that a GPU seldom takes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"

pytestmark = pytest.mark.skipif(not os.path.exists(CLANG), reason="clang++ not available")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kernels") / "host_expert_kernels")
    native = os.path.join(ROOT, "tests", "native")
    # -fwrapv: whole numbers that pass their range wrap, as on the GPU
    cmd = [CLANG, "-std=c++17", "-O1", "-g", "-fwrapv", "-I", os.path.join(native, "lanes"), "-I", os.path.join(ROOT, "include"),
           os.path.join(native, "host_expert_kernels.cpp"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    return exe


@pytest.mark.parametrize("what", ["in_place", "sort", "far"])
def test_kernels(program, what):
    res = subprocess.run([program, what], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "0 failures" in res.stdout, res.stdout + res.stderr[-4000:]
