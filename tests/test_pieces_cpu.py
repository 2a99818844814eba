"""csrc/pieces.h, the arithmetic that places a workgroup's lanes in rows, on the host."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_every_number_of_pieces_a_row(tmp_path, host_only):
    exe = tmp_path / "pieces"
    cmd = ["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "concurrent_gemm_dma_amd", "csrc"),
           os.path.join(ROOT, "tests", "pieces_main.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
