"""The vector verbs on the host alone (no device): their launch plans under the
sanitizers, the refusals of their C entry points, and the binding's argument
checks that come before any device call."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "histogram_gradient_boosted_amd")
SOURCE = os.path.join(ROOT, "tests", "host", "vector_test.cpp")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g"]


def _run(exe, what, **env):
    r = subprocess.run([exe, what], capture_output=True, text=True, timeout=300, env=dict(os.environ, **env))
    assert r.returncode == 0 and "checks passed" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_plans_under_sanitizers(tmp_path):
    exe = str(tmp_path / "vector_test")
    subprocess.run(["g++", "-std=c++17", "-O1", *SAN, "-I", os.path.join(PKG, "csrc"), "-o", exe, SOURCE], check=True)
    _run(exe, "plan", ASAN_OPTIONS="detect_leaks=1:abort_on_error=0")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_c_entry_points_refuse_bad_arguments(tmp_path):
    if not os.path.exists(os.path.join(PKG, "libhgb.so")):
        pytest.fail("libhgb.so not built: run __graft_entry__.build()")
    exe = str(tmp_path / "vector_test")
    subprocess.run(["g++", "-std=c++17", "-O1", "-DWITH_LIBRARY", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(PKG, "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", "-o", exe, SOURCE,
                    "-L", PKG, "-l:libhgb.so", "-L", "/opt/rocm/lib", "-lamdhip64",
                    f"-Wl,-rpath,{PKG}:/opt/rocm/lib"], check=True)
    _run(exe, "refusals")


def test_binding_refuses_host_tensors():
    import torch

    from histogram_gradient_boosted_amd import binding
    ctx = binding.Context.__new__(binding.Context)   # no device: only the checks run
    ctx._torch, ctx._lib, ctx.device = torch, binding.load(), 0
    ctx._types = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    r = binding.Route(i.reshape(-1), i, torch.zeros(4, dtype=torch.int32))
    for call in (lambda: ctx.embed(x, i), lambda: ctx.embed_backward(x, i[:, 0], 5), lambda: ctx.layer_norm(x),
                 lambda: ctx.layer_norm_backward(x, x, x[:, 0], x[:, 0]), lambda: ctx.route(i, 3),
                 lambda: ctx.route_gather(x, r), lambda: ctx.route_combine(x, r), lambda: ctx.route_gather_backward(x, r),
                 lambda: ctx.route_combine_backward(x, x, r)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
