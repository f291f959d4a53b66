"""The gate and the head's losses on the host alone (no device): their plans
under the sanitizers, the refusals of their C entry points, the launches that
they ask for, and the binding's checks that come before any device call."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "histogram_gradient_boosted_amd")
SOURCE = os.path.join(ROOT, "tests", "host", "head_test.cpp")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g"]

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")


def run(exe, what, **env):
    r = subprocess.run([exe, what], capture_output=True, text=True, timeout=300, env=dict(os.environ, **env))
    assert r.returncode == 0 and "checks passed" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


def test_plans_under_sanitizers(tmp_path):
    exe = str(tmp_path / "head_test")
    subprocess.run(["g++", "-std=c++17", "-O1", *SAN, "-I", os.path.join(PKG, "csrc"), "-o", exe, SOURCE], check=True)
    run(exe, "plan", ASAN_OPTIONS="detect_leaks=1:abort_on_error=0")


def test_plans_of_three_planes_under_sanitizers(tmp_path):
    exe = str(tmp_path / "head_test")
    subprocess.run(["g++", "-std=c++17", "-O1", *SAN, "-I", os.path.join(PKG, "csrc"), "-o", exe, SOURCE], check=True)
    run(exe, "planes", ASAN_OPTIONS="detect_leaks=1:abort_on_error=0")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(os.path.join(PKG, "libhgb.so")):
        pytest.fail("libhgb.so not built: run __graft_entry__.build()")
    exe = str(tmp_path_factory.mktemp("head") / "head_test")
    subprocess.run(["g++", "-std=c++17", "-O1", "-DWITH_LIBRARY", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(PKG, "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", "-o", exe, SOURCE,
                    "-L", PKG, "-l:libhgb.so", "-L", "/opt/rocm/lib", "-lamdhip64",
                    f"-Wl,-rpath,{PKG}:/opt/rocm/lib"], check=True)
    return exe


def test_c_entry_points_refuse_bad_arguments(program):
    run(program, "refusals")


def test_every_accepted_size_fits_a_launch(program):
    run(program, "grids")


def test_gradients_of_no_rows_fit_a_launch(program):
    run(program, "no_rows")


def test_factors_that_overflow_in_the_kernels_are_refused(program):
    run(program, "factors")


@pytest.fixture()
def ctx():
    import torch

    from histogram_gradient_boosted_amd import binding
    c = binding.Context.__new__(binding.Context)   # no device: only the checks run
    c._torch, c._lib, c.device = torch, binding.load(), 0
    return c


def calls(ctx, x):
    """Every verb, given x ([4, 8]) as its vectors."""
    import torch
    i, one = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    s = torch.zeros(4, 2, dtype=torch.int32)
    return (lambda: ctx.gate(x, 2), lambda: ctx.gate_backward(one, x, s), lambda: ctx.cross_entropy(x, x, i),
            lambda: ctx.cross_entropy_backward(one, x, x, i, one), lambda: ctx.distill(x, x, s, x[:, :2]),
            lambda: ctx.distill_backward(one, x, x, s, x[:, :2], one, x[:, :2]))


def test_binding_refuses_host_tensors(ctx):
    import torch
    for call in calls(ctx, torch.zeros(4, 8)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_binding_refuses_what_torch_would_lose(ctx):
    import torch
    for call in calls(ctx, torch.zeros(4, 8, requires_grad=True)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    x = torch.ones(4, 8, dtype=torch.complex64).conj().imag
    assert x.is_neg()
    for call in calls(ctx, x):
        with pytest.raises(ValueError, match="resolve_neg"):
            call()
