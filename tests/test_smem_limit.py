"""The kernels' shared-memory limit under calls of several host threads (no
GPU): no call lowers it under another's launch."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_first_calls_of_two_threads(tmp_path):
    from sparse_attention_decode_paged_gb300 import build

    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path / "smem_limit_host"
    cmd = [cxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-Wno-unused-parameter",
           "-I", os.path.join(build.cuda_home(), "include"), "-I", build.CSRC, "-I", build.INCLUDE,
           os.path.join(ROOT, "tests", "smem_limit_host.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok"
