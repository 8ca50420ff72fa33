"""The feed-forward C ABI layer under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU.

ffn_abi.cpp is compiled with g++ (host code only) together with
tests/ffn_abi_host_stub.cpp, which stands in for the kernel launchers.  The
argument checks of tests/test_ffn_abi.py and tests/test_ffn_abi_ranges.py then run
in a child process against that library, with libasan preloaded, and so does
tests/test_ffn_abi_dispatch.py.  Any sanitizer report fails the child, and so this
test.
"""

import os
import subprocess
import sys

import pytest

from tests.test_abi_sanitized import CSRC, ROCM_INCLUDE, ROOT, SANITIZE, _tool

# The package's __init__ and torch stay out of the sanitized process: the library
# modules alone are loaded, and the default library is the host-stub build.
RUNNER = r"""
import os, sys, types
root = sys.argv[1]
sys.path.insert(0, root)
pkg = types.ModuleType("fp8_block_scaled_quant_amd")
pkg.__path__ = [os.path.join(root, "fp8_block_scaled_quant_amd")]
sys.modules["fp8_block_scaled_quant_amd"] = pkg
sys.modules["torch"] = types.ModuleType("torch")
from fp8_block_scaled_quant_amd import _ffn_lib
_ffn_lib.LIB_PATH = os.environ["FP8BSQ_FFN_TEST_LIB"]
import pytest
tests = [os.path.join(root, "tests", "test_ffn_abi" + name + ".py") for name in ("", "_ranges", "_dispatch")]
sys.exit(pytest.main(["-q", "-p", "no:cacheprovider", "-rs", "-k", "not python_functions", *tests]))
"""


@pytest.fixture(scope="module")
def stub_lib(tmp_path_factory):
    gxx = _tool("g++")
    if not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("HIP headers not found")
    out = str(tmp_path_factory.mktemp("ffn_abi_asan") / "libfp8bsq_ffn_hoststub.so")
    cmd = [gxx, "-std=c++17", "-O1", "-g", *SANITIZE, "-fPIC", "-shared", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__",
           "-I", ROCM_INCLUDE, "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "ffn_abi.cpp"),
           os.path.join(ROOT, "tests", "ffn_abi_host_stub.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return out


def test_ffn_abi_under_asan_and_ubsan(stub_lib):
    asan = subprocess.run([_tool("g++"), "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("libasan not found")
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", FP8BSQ_FFN_TEST_LIB=stub_lib)
    r = subprocess.run([sys.executable, "-c", RUNNER, ROOT], capture_output=True, text=True, env=env, timeout=600)
    text = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in text and "runtime error:" not in text, text
    assert r.returncode == 0, text
    # the dispatch checks ran (they skip against the real library)
    assert "skipped" not in r.stdout.splitlines()[-1], text
