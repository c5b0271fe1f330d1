"""muonh_step_quantized refuses outputs inside the handle's workspace: its host
code built with g++ under AddressSanitizer and UndefinedBehaviorSanitizer and
driven with no device, and the library's own workspace on a GPU."""

import os
import shutil
import subprocess

import pytest
import torch

import pretraining_optimizer_amd as pm

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "pretraining_optimizer_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="g++ or the ROCm headers are missing")
def test_outputs_in_the_workspace_are_refused(tmp_path):
    exe = tmp_path / "step_workspace_driver"
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
             "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
             "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"]
    srcs = [os.path.join(CSRC, "operators.cpp"), os.path.join(CSRC, "step_fp8.cpp"),
            os.path.join(HERE, "host_sanitize", "step_workspace_driver.cpp")]
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


@pytest.mark.gpu
def test_a_handle_with_the_callers_workspace():
    """The refusal through the library, and that a step whose outputs lie outside
    runs: in a workspace of the caller's, its outputs right behind it."""
    w, m, g = (torch.randn((200, 130), device="cuda") for _ in range(3))
    need = pm.workspace_size([(200, 130)], g_dtype=pm.MUONH_F32)
    need = -(-need // 256) * 256
    memory = torch.zeros(need + 256 * 512 + 4096, dtype=torch.uint8, device="cuda")
    opt = pm.MuonH([w], [m], grad_dtype=torch.float32, workspace=memory.data_ptr(), workspace_bytes=need)

    def form(at):
        data = memory[at:at + 200 * 256].view(200, 256).view(torch.float8_e4m3fn)
        return pm.Fp8Matrix(data, memory[-64:-56].view(2, 4), 130, 128)

    keep = w.clone()
    for at in (0, need - 256):
        with pytest.raises(pm.MuonHError, match="workspace"):
            opt.step([g], elr=0.01, fp8=[(form(at), None)])
    torch.cuda.synchronize()
    assert torch.equal(w, keep)
    q = form(need)
    opt.step([g], elr=0.01, fp8=[(q, None)])
    ref = pm.fp8_quantize(w, block_rows=128)
    assert not torch.equal(w, keep)
    assert torch.equal(q.data.view(torch.uint8), ref.data.view(torch.uint8)) and torch.equal(q.scale, ref.scale)
    opt.close()
