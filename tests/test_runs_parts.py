"""Sizes that the launch of long runs works out on the host, in a host-only build under UndefinedBehaviorSanitizer (CPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tokens_of_a_tile(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    stubs = os.path.join(ROOT, "tests", "sanitize")
    exe = str(tmp_path / "seen_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", stubs, "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "bit_ptq_reconstruction_amd", "csrc"),
                    os.path.join(stubs, "seen_check.cpp"), "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
