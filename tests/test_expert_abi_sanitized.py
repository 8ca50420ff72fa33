"""The expert operators' C ABI layer under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: ffn_abi.cpp over stand-ins for all launchers
(expert_abi_host_stub.cpp), driven by test_expert_abi.py and
test_expert_abi_dispatch.py in a child process.  Any report fails it."""

import os
import subprocess
import sys

import pytest

from tests.test_abi_sanitized import CSRC, ROCM_INCLUDE, ROOT, SANITIZE, _tool

# torch and the package's __init__ stay out of the sanitized process
RUNNER = r"""
import os, sys, types
root = sys.argv[1]
sys.path.insert(0, root)
pkg = types.ModuleType("fp8_block_scaled_quant_amd")
pkg.__path__ = [os.path.join(root, "fp8_block_scaled_quant_amd")]
sys.modules["fp8_block_scaled_quant_amd"] = pkg
sys.modules["torch"] = types.ModuleType("torch")
from fp8_block_scaled_quant_amd import _ffn_lib
_ffn_lib.LIB_PATH = os.environ["FP8BSQ_EXPERT_TEST_LIB"]
import pytest
tests = [os.path.join(root, "tests", "test_expert_abi" + name + ".py") for name in ("", "_dispatch")]
sys.exit(pytest.main(["-q", "-p", "no:cacheprovider", "-rs", "-k", "not python_functions", *tests]))
"""


@pytest.fixture(scope="module")
def stub_lib(tmp_path_factory):
    gxx = _tool("g++")
    if not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("HIP headers not found")
    out = str(tmp_path_factory.mktemp("expert_abi_asan") / "libfp8bsq_expert_hoststub.so")
    cmd = [gxx, "-std=c++17", "-O1", "-g", *SANITIZE, "-fPIC", "-shared", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "ffn_abi.cpp"),
           os.path.join(ROOT, "tests", "expert_abi_host_stub.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return out


def test_expert_abi_under_asan_and_ubsan(stub_lib):
    asan = subprocess.run([_tool("g++"), "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("libasan not found")
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", FP8BSQ_EXPERT_TEST_LIB=stub_lib)
    r = subprocess.run([sys.executable, "-c", RUNNER, ROOT], capture_output=True, text=True, env=env, timeout=600)
    text = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in text and "runtime error:" not in text, text
    assert r.returncode == 0, text
    assert "skipped" not in r.stdout.splitlines()[-1], text   # the dispatch checks ran
