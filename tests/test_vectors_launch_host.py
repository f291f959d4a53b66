"""What the vector verbs' entry points ask of the runtime, checked on the host
alone: the test program stands in for the runtime's launch functions."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "histogram_gradient_boosted_amd")
SOURCE = os.path.join(ROOT, "tests", "host", "vector_launch_test.cpp")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    if not os.path.exists(os.path.join(PKG, "libhgb.so")):
        pytest.fail("libhgb.so not built: run __graft_entry__.build()")
    exe = str(tmp_path_factory.mktemp("launch") / "vector_launch_test")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(PKG, "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", "-o", exe, SOURCE,
                    "-L", PKG, "-l:libhgb.so", "-L", "/opt/rocm/lib", "-lamdhip64",
                    f"-Wl,-rpath,{PKG}:/opt/rocm/lib"], check=True)
    return exe


def run(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "checks passed" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


def test_every_accepted_size_fits_a_launch(program):
    run(program, "grids")


def test_arguments_side_by_side_in_one_buffer_are_taken(program):
    run(program, "apart")


def test_contexts_do_not_lower_each_other_s_lds(program):
    run(program, "contexts")
