"""Which kernel an int8 product takes, on the host: the shapes that the GPU tests run reach every kernel,
with results of both types, and both ways of the last round."""
import os
import shutil
import subprocess

import pytest

import test_gpu_i8 as shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = {"rounds 4", "rounds 8", "128x128 two", "128x128", "128x64", "64x64", "64x32"} | {
    f"{rows} by {waves}" for rows in (16, 32) for waves in (1, 2, 4, 8)}


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    exe = tmp_path_factory.mktemp("choice") / "choice"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "concurrent_gemm_dma_amd", "csrc"),
                        os.path.join(ROOT, "tests", "i8_choice_main.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60)
        lines = [line.split(",") for line in r.stdout.splitlines()]
        assert r.returncode == 0 and len(lines) == len(cases)
        return [(name, q == "1") for name, q in lines]

    return run


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_the_gpu_tests_reach_every_kernel(host_only, choose):
    one = [(M, N, K, 1, 0, f32) for M, N, K in shapes.EVERY for f32 in (0, 1)]
    experts = [(M, N, K, E, 1, i % 2) for i, (M, E, N, K) in enumerate(shapes.EVERY_EXPERTS)]
    got = choose(one + experts)
    assert {(k, c[5]) for (k, _), c in zip(got, one + experts)} == {(k, f32) for k in KERNELS for f32 in (0, 1)}
    for kernel in ("rounds 4", "rounds 8"):
        assert {q for k, q in got[:len(one)] if k == kernel} == {False, True}
    # and with experts, where the device counts the tiles
    assert {"rounds 4", "rounds 8"} <= {k for k, _ in got[len(one):]}


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_choices_that_the_measurements_stand_for(host_only, choose):
    """Shapes whose times with several kernels stand beside the model or the kernels."""
    want = {(1, 28672, 8192): "16 by 4", (198, 3055, 2199): "64x64", (300, 4096, 4096): "128x64", (1024, 4096, 4096): "128x128",
            (8192, 28672, 8192): "rounds 4", (8192, 28672, 512): "rounds 8", (128, 4096, 14336): "64x32"}
    got = choose([(M, N, K, 1, 0, 0) for M, N, K in want])
    assert {shape: k for shape, (k, _) in zip(want, got)} == want
