"""Entry points run on the device the library was bound to, whichever one is current, and leave that
one current; on the host, with HIP's device calls and all launches replaced."""
import os
import shutil
import subprocess

import pytest

from concurrent_gemm_dma_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_calls_run_on_the_library_s_device(tmp_path, host_only):
    exe = tmp_path / "device"
    cmd = ["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", build.INCLUDE, "-I", build.CSRC,
           "-I", os.path.join(build.ROCM, "include"), os.path.join(ROOT, "tests", "device_main.cpp"),
           os.path.join(build.CSRC, "layer.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
