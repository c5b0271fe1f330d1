"""What muonh_step_quantized keeps between steps, driven on the host with HIP as a
stub (CPU only, under AddressSanitizer and UndefinedBehaviorSanitizer): failed
calls leave nothing behind, changed outputs are uploaded, unchanged ones not."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "pretraining_optimizer_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="g++ or the ROCm headers are missing")
def test_tables_of_the_quantised_step(tmp_path):
    exe = tmp_path / "step_tables_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           os.path.join(CSRC, "operators.cpp"), os.path.join(CSRC, "step_fp8.cpp"),
           os.path.join(HERE, "host_sanitize", "step_tables_driver.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "all checks passed" in out, out[-4000:]
    assert "runtime error" not in out and "Sanitizer" not in out, out[-4000:]
