"""Kernels run on the host: the experts' with a fiber for each lane, in orders that a GPU seldom takes, and the rotary
positions' sines and cosines."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"

pytestmark = pytest.mark.skipif(not os.path.exists(CLANG), reason="clang++ not available")


def build(folder, name):
    exe, native = str(folder / name), os.path.join(ROOT, "tests", "native")
    # -fwrapv: whole numbers that pass their range wrap, as on the GPU
    cmd = [CLANG, "-std=c++17", "-O1", "-g", "-fwrapv", "-I", os.path.join(native, "lanes"), "-I", os.path.join(ROOT, "include"),
           "-x", "c++", os.path.join(native, name + ".cpp"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    return exe


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return build(tmp_path_factory.mktemp("kernels"), "host_expert_kernels")


@pytest.mark.parametrize("what", ["in_place", "sort", "far"])
def test_kernels(program, what):
    res = subprocess.run([program, what], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "0 failures" in res.stdout, res.stdout + res.stderr[-4000:]


def test_sines_and_cosines(tmp_path):
    res = subprocess.run([build(tmp_path, "host_rotary_turn")], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "0 failures" in res.stdout, res.stdout + res.stderr[-4000:]
