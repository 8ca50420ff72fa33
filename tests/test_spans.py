"""The test for tensors that share memory, against every pair of spans, under
AddressSanitizer and UndefinedBehaviorSanitizer (host code only)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is needed to build the check")
def test_overlaps_match_every_pair(tmp_path):
    exe = str(tmp_path / "spans_check")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall",
                        "-I", os.path.join(ROOT, "fp8_block_scaled_quant_amd", "csrc"),
                        os.path.join(ROOT, "tests", "spans_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
