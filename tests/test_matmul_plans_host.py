"""How the FP8 product runs at the sizes that the GPU tests use, checked on the
host (CPU only): each tile kernel, whole and split, has a size that takes it."""

import os
import shutil
import subprocess

import pytest

import test_gpu_block_fp8
from matmul_plans import KERNELS, TILES

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
    for (bf16, f32), sizes in KERNELS.items():
        for result, want in (("bf16", bf16), ("f32", f32)):
            for size, p in zip(sizes, plans([(*s, *blocks, result) for s in sizes])):
                tile = f"{64 * p[0]}x{64 * p[1]}" + (" split" if p[2] > 1 else "")
                kernel = tile if p[0] else "direct" if p[4] else "narrow"
                assert kernel == want, (size, result)


def test_every_size_of_the_gpu_tests_is_pinned():
    pinned = {size for sizes in KERNELS.values() for size in sizes}
    tested = test_gpu_block_fp8.SHAPES + test_gpu_block_fp8.NARROW + [(n, m, k) for m, n, k in test_gpu_block_fp8.NARROW]
    for name in ("test_matmul_tiles_ragged", "test_matmul_accumulate_and_pitch", "test_two_products_at_once_and_two_graphs"):
        marks = getattr(test_gpu_block_fp8, name).pytestmark
        tested += [size for m in marks if m.name == "parametrize" and m.args[0] == "m,n,k" for size in m.args[1]]
    assert set(tested) <= pinned


def test_every_tile_that_a_product_takes_is_tested(plans):
    sizes = [17, 33, 48, 65, 100, 129, 200, 300, 401, 640, 777, 1000, 1500, 2048, 2500, 5000, 8192, 12288, 16384, 32768]
    lengths = [100, 384, 640, 1100, 1500, 2048, 6144, 8192, 9000, 16384, 30000, 65536]
    cases = [(m, n, k, 1, 1, t) for m in sizes for n in sizes for k in lengths for t in ("bf16", "f32")]
    taken = {(ma, nb, s > 1, c[5]) for c, (ma, nb, s, _, _) in zip(cases, plans(cases)) if ma}
    assert taken == {(p[0], p[1], p[2] > 1, t) for _, _, _, t, p in TILES}
