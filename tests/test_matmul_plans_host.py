"""How the FP8 product runs at the sizes that the GPU tests use, checked on the
host (CPU only): each tile kernel, whole and split, has a size that takes it."""

import os
import shutil
import subprocess

import pytest

from matmul_plans import OTHERS, TILES

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                                reason="g++ or the ROCm headers are missing")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = tmp_path_factory.mktemp("plans") / "matmul_plans"
    cmd = ["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "pretraining_optimizer_amd", "csrc", "operators.cpp"),
           os.path.join(HERE, "host_plan", "matmul_plans.cpp"), "-o", str(exe), "-L", os.path.join(ROCM, "lib"),
           "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(cases):
        """(ma, nb, splits, split_blocks, direct) of each (m, n, k, block_a, block_b, result)."""
        text = "\n".join(" ".join(str(v) for v in (*c[:5], int(c[5] == "bf16"))) for c in cases)
        r = subprocess.run([str(exe)], input=text + "\n", capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr[-4000:]
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]

    return run


@pytest.mark.parametrize("blocks", [(1, 1), (1, 128), (128, 1), (128, 128)])
def test_plans_of_the_tested_sizes(plans, blocks):
    got = plans([(m, n, k, *blocks, t) for m, n, k, t, _ in TILES])
    assert [g[:4] for g in got] == [want for *_, want in TILES]
    got = plans([(m, n, k, *blocks, t) for m, n, k, t, _ in OTHERS])
    assert [(g[0], g[1], g[2] > 1, g[4] == 1) for g in got] == [want for *_, want in OTHERS]


def test_every_tile_that_a_product_takes_is_tested(plans):
    sizes = [17, 33, 48, 65, 100, 129, 200, 300, 401, 640, 777, 1000, 1500, 2048, 2500, 5000, 8192, 12288, 16384, 32768]
    lengths = [100, 384, 640, 1100, 1500, 2048, 6144, 8192, 9000, 16384, 30000, 65536]
    cases = [(m, n, k, 1, 1, t) for m in sizes for n in sizes for k in lengths for t in ("bf16", "f32")]
    taken = {(ma, nb, s > 1, c[5]) for c, (ma, nb, s, _, _) in zip(cases, plans(cases)) if ma}
    assert taken == {(p[0], p[1], p[2] > 1, t) for _, _, _, t, p in TILES}
