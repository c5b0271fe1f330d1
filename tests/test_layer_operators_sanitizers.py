"""The host code of the attention, the residual norm and the embedding built with g++
under AddressSanitizer and UndefinedBehaviorSanitizer and driven with no device:
workspaces, refusals, empty calls, what the launchers are given (CPU only)."""

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
def test_layer_operators_host_code_under_asan_ubsan(tmp_path):
    exe = tmp_path / "layer_operators_driver"
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
             "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
             "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"]
    srcs = [os.path.join(CSRC, f) for f in ("operators.cpp", "attention.cpp", "add_norm.cpp", "embedding.cpp")]
    srcs.append(os.path.join(HERE, "host_sanitize", "layer_operators_driver.cpp"))
    cmd = ["g++", *flags, *srcs, "-o", str(exe), "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
           f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    supp = tmp_path / "lsan.supp"
    supp.write_text("leak:libamdhip64\nleak:libhsa-runtime64\nleak:libdrm\nleak:librocprofiler\n")
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:halt_on_error=1",
               LSAN_OPTIONS=f"suppressions={supp}", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "all checks passed" in out, out[-4000:]
    assert "runtime error" not in out and "Sanitizer" not in out, out[-4000:]
