"""What the training-step operators launch, seen without a GPU: a program that stands in for the runtime's
launch functions calls libtide_step.so with made-up addresses."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "all_gather_placement_amd")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("launches") / "host_step_launches")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "host_step_launches.cpp"),
           "-rdynamic", "-L" + PKG, "-l:libtide_step.so", "-Wl,-rpath," + PKG, "-L/opt/rocm/lib",
           "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    return exe


@pytest.mark.parametrize("what", ["sort", "columns", "far", "scalars", "blocks", "parts", "failed", "stale"])
def test_launches(program, what):
    res = subprocess.run([program, what], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "0 failures" in res.stdout, res.stdout + res.stderr[-4000:]
