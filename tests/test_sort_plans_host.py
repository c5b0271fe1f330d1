"""How the embedding gradient orders the tokens of the sizes that the GPU tests use, checked
on the host (CPU only): every path has sizes that take it, on both sides of each limit."""

import os
import shutil
import subprocess

import pytest

from sort_plans import SORTS

HERE = os.path.dirname(os.path.abspath(__file__))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="g++ or the ROCm headers are missing")
def test_sorts_of_the_tested_sizes(tmp_path):
    exe = tmp_path / "sort_plans"
    cmd = ["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           os.path.join(HERE, "host_plan", "sort_plans.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    text = "\n".join(f"{n} {rows}" for n, rows, *_ in SORTS)
    r = subprocess.run([str(exe)], input=text + "\n", capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-4000:]
    got = [line.split() for line in r.stdout.splitlines()]
    assert [(int(p), int(b), path) for p, b, path in got] == [(p, b, path) for _, _, p, b, path in SORTS]
    assert {(p, path) for _, _, p, _, path in SORTS if path != "ranked"} == {
        (p, path) for p in (1, 2, 3, 4) for path in ("own", "begin")}
